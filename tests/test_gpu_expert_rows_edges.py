"""The rows' way out and back where a kernel changes its form: products beyond
fp32's range in the K-grouped scatter, more blocks of rows than a grid axis,
masked buffers of many rows, weight gradients over groups of eight choices, and
layouts whose counts go through the workspace."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

KEEP = 0xA5                      # code left where nothing may be written


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def exact_codes(x, amax):
    """e4m3 values of x * 448 / amax rounded to nearest even, in whole numbers: x bf16 values and amax
    bf16 values > 0, fp64 arrays that broadcast; also where a quotient lies halfway between two codes."""
    x, amax = np.broadcast_arrays(x, amax)
    fx, ex = np.frexp(np.abs(x))
    fa, ea = np.frexp(amax)
    mx, ma = (fx * 256).astype(np.int64), (fa * 256).astype(np.int64)         # 8 bits each
    d = ex.astype(np.int64) - ea                                              # q = 448 * mx / ma * 2^d
    live = (mx > 0) & (d > -24)
    d = np.where(live, d, 0)
    e = np.full(x.shape, -6, dtype=np.int64)                                  # q's binade, at least e4m3's lowest
    for b in range(-5, 9):                                                    # q >= 2^b
        up, down = np.maximum(d - b, 0), np.maximum(b - d, 0)
        e = np.where(448 * mx << up >= ma << down, b, e)
    sh = d - (e - 3)                                                          # steps: 448 * mx * 2^sh / ma
    num, den = 448 * mx << np.maximum(sh, 0), ma << np.maximum(-sh, 0)
    n, rest = num // den, num % den
    tie = live & (2 * rest == den)
    n = n + ((2 * rest > den) | (tie & (n % 2 == 1)))
    return np.where(live, np.sign(x) * np.ldexp(n.astype(np.float64), e - 3), 0.0), tie


@pytest.mark.parametrize("form", ["contiguous", "k-grouped"])
def test_codes_are_the_nearest_in_exact_arithmetic(dg, form):
    # bf16 blocks hold quotients x / (amax / 448) that lie exactly halfway between two codes, and
    # those go to the even one: whole numbers decide, so every code has to be equal
    print(f"case: {form} scatter against exact quotients", flush=True)
    rng = np.random.default_rng(16)
    M, K = 1024, 1024
    x = (rng.standard_normal((M, K)) * np.exp(0.5 * rng.standard_normal((1, K)))).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16)
    rows = torch.arange(M, dtype=torch.int32, device="cuda")
    a = torch.full((M, K), KEEP, dtype=torch.uint8, device="cuda")
    v = x.double().numpy()
    if form == "contiguous":
        sfa = torch.empty(K // 128, M, device="cuda")
        dg.dg_m_grouped_scatter_fp8_contiguous(x.cuda(), None, rows.view(M, 1), rows, a, sfa)
        blocks = v.reshape(M, K // 128, 128)
        want, tie = exact_codes(blocks, np.abs(blocks).max(axis=2, keepdims=True))
    else:
        sfa = torch.empty(M // 128, K, device="cuda")
        dg.dg_k_grouped_scatter_fp8(x.cuda(), None, rows, 1, a, sfa)
        blocks = v.reshape(M // 128, 128, K)
        want, tie = exact_codes(blocks, np.abs(blocks).max(axis=1, keepdims=True))
    torch.cuda.synchronize()
    assert tie.sum() > 1000
    got = oracle.decode_e4m3(a.cpu().numpy()).astype(np.float64)
    assert np.array_equal(got, want.reshape(M, K))
