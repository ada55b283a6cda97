"""The rows' way out and back where a kernel changes its form: products beyond
fp32's range in the K-grouped scatter, more blocks of rows than a grid axis,
masked buffers of many rows, weight gradients over groups of eight choices, and
layouts whose counts go through the workspace."""
import numpy as np
import pytest
import torch

import oracle
from oracle import around
from tests.gpu_util import dev

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


def i32(*shape, fill=-9):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def is_nan_code(c):
    return (c & 0x7F) == 0x7F


def check_block_codes(codes, sf, v, amax, pow2):
    """codes and sf of the fp64 values v with block maxima amax (sf broadcasts to v)."""
    want = around.block_scales(amax, pow2)
    # one rounding to fp32; a power of two is exact
    assert np.all(np.abs(sf - want) <= (0.0 if pow2 else 2.0 ** -23) * want)
    u = v / sf
    q = oracle.decode_e4m3(codes).astype(np.float64)
    # the nearest code, and the roundings of the quotient (2^-24 each) before it
    near = 0.5 * around.e4m3_step(u) + 4 * 2.0 ** -24 * np.abs(u)
    assert np.all(np.abs(q - np.clip(u, -448.0, 448.0)) <= near)


@pytest.mark.parametrize("pow2", [False, True])
def test_kgrouped_scatter_of_products_beyond_fp32(dg, pow2):
    # weight times value may exceed the largest fp32 value, and their scale not: 1.5e41 / 448 is
    # the most; columns with such a product beside ordinary ones
    print(f"case: K-grouped scatter of products up to 1e41, pow2={pow2}", flush=True)
    rng = np.random.default_rng(11)
    T, N = 300, 160
    x = rng.standard_normal((T, N)).astype(np.float32)
    x[:, ::3] *= np.float32(2.0 ** 126)
    x = torch.from_numpy(np.clip(x, -3e38, 3e38)).to(torch.bfloat16)
    w = (rng.random((T, 1)) * 100.0 + 1.0).astype(np.float32)
    w[5::7] *= np.float32(1e-3)
    K = 384
    slot = np.full(K, -1, dtype=np.int32)
    slot[:T] = rng.permutation(T)
    a = torch.full((K, N), KEEP, dtype=torch.uint8, device="cuda")
    sfa = torch.full((K // 128, N), -3.0, device="cuda")
    dg.dg_k_grouped_scatter_fp8(x.cuda(), dev(w), dev(slot), 1, a, sfa, pow2_scales=pow2)
    torch.cuda.synchronize()
    v = np.where(slot[:, None] >= 0, x.double().numpy()[slot] * w.astype(np.float64)[slot], 0.0).reshape(K // 128, 128, N)
    amax = np.abs(v).max(axis=1)
    assert amax.max() > 3.5e38 and amax.max() < 1.4e41
    codes = a.cpu().numpy()
    assert not is_nan_code(codes).any()
    check_block_codes(codes.reshape(v.shape), sfa.cpu().numpy().astype(np.float64)[:, None, :], v, amax[:, None, :], pow2)


@pytest.mark.parametrize("weighted", [False, True])
def test_kgrouped_scatter_of_nonfinite_values(dg, weighted):
    # as in the M-grouped forms: a NaN keeps to its place, an infinity makes its block's scale infinite
    print(f"case: K-grouped scatter of NaN and infinities, weighted={weighted}", flush=True)
    x = torch.ones(4, 32, dtype=torch.bfloat16)
    x[0, 3], x[1, 5], x[2, 9] = float("nan"), float("inf"), float("-inf")
    x[:, 20] = float("nan")
    slot = np.full(128, -1, dtype=np.int32)
    slot[[0, 7, 64, 127]] = [0, 1, 2, 3]
    w = torch.full((4, 1), 2.0, device="cuda") if weighted else None
    a = torch.zeros(128, 32, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(1, 32, device="cuda")
    dg.dg_k_grouped_scatter_fp8(x.cuda(), w, dev(slot), 1, a, sfa)
    torch.cuda.synchronize()
    c, s = a.cpu().numpy(), sfa.cpu().numpy()[0]
    nan = is_nan_code(c)
    assert nan[0, 3] and nan[7, 5] and nan[64, 9] and nan[[0, 7, 64, 127], 20].all() and nan.sum() == 7
    assert np.isinf(s[[5, 9]]).all() and s[20] == 1.0 and s[3] == np.float32((2.0 if weighted else 1.0) / 448.0)
    assert np.all(c[[7, 64, 127], 3] == 0x7E) and np.all(c[1:7] == 0) and np.all(c[[0, 64, 127], 5] == 0)


def test_kgrouped_scatter_of_more_blocks_than_a_grid_axis(dg):
    print("case: K-grouped scatter of 65539 blocks of rows", flush=True)
    rng = np.random.default_rng(12)
    K, N, T = 65539 * 128, 32, 6
    x = bf16(rng, T, N)
    rows = torch.tensor([0, 65534 * 128 + 127, 65535 * 128, 65536 * 128 + 5, K - 129, K - 1])
    slot = torch.full((K,), -1, dtype=torch.int32)
    slot[rows] = torch.arange(T, dtype=torch.int32)
    a = torch.full((K, N), KEEP, dtype=torch.uint8, device="cuda")
    sfa = torch.full((K // 128, N), -3.0, device="cuda")
    dg.dg_k_grouped_scatter_fp8(x.cuda(), None, slot.cuda(), 1, a, sfa)
    torch.cuda.synchronize()
    block = torch.div(rows, 128, rounding_mode="floor")
    assert len(set(block.tolist())) == T                  # one row each: its own maximum
    v = x.double().numpy()
    check_block_codes(a[rows.cuda()].cpu().numpy(), sfa[block.cuda()].cpu().numpy().astype(np.float64), v, np.abs(v), False)
    assert int((a != 0).any(1).sum()) == T
    sfa[block.cuda()] = 1.0
    assert bool((sfa == 1.0).all())                       # blocks without a choice


WGRAD = [
    # T, top_k, M, N: from 512 tokens on and more than two choices, eight to a workgroup
    (512, 3, 700, 129), (513, 8, 900, 2047), (700, 11, 400, 520), (600, 64, 300, 77), (2050, 4, 1000, 4096), (900, 9, 50, 3),
]


@pytest.mark.parametrize("shape", WGRAD, ids=str)
def test_gather_weight_gradient_by_eights(dg, shape):
    T, k, M, N = shape
    print(f"case: gather weight gradient {shape}", flush=True)
    rng = np.random.default_rng(N + T)
    rows, g = bf16(rng, M, N), bf16(rng, T, N)
    at = rng.integers(0, M, (T, k)).astype(np.int32)
    at[rng.random((T, k)) < 0.2] = -1
    at[0, -1] = M
    at[1] = -1
    at[2, :-1] = -1
    out = torch.full((T, k), float("nan"), device="cuda")
    dg.dg_m_grouped_gather_weight_grad(rows.cuda(), dev(at), g.cuda(), out)
    torch.cuda.synchronize()
    ref, mag = around.gather_weight_grad(rows.float().numpy(), at, g.float().numpy())
    # products of bf16 are exact in fp32; N additions in any order
    assert np.all(np.abs(out.cpu().numpy() - ref) <= N * 2.0 ** -24 * mag + 1e-37)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_masked_scatter_into_many_rows(dg, weighted, pow2):
    # from 32768 rows on the scales are written row by row, here into [G][K/128][max_m]
    G, max_m, T, k, K = 130, 300, 700, 3, 384
    print(f"case: masked scatter into {G} x {max_m} rows, weighted={weighted} pow2={pow2}", flush=True)
    rng = np.random.default_rng(13)
    ids = np.stack([rng.permutation(G)[:k] for _ in range(T)]).astype(np.int32)
    ids[:400, 0] = 7                                      # one expert runs over
    ids[:400, 1:] = np.stack([rng.permutation(G - 8)[:k - 1] + 8 for _ in range(400)])
    x = bf16(rng, T, K)
    w = (rng.random((T, k)).astype(np.float32) - 0.3) if weighted else None
    masked_m, row_of, slot_of = i32(G), i32(T, k), i32(G, max_m)
    dg.dg_m_grouped_layout_masked(dev(ids), 0, masked_m, row_of, slot_of)
    a = torch.full((G, max_m, K), KEEP, dtype=torch.uint8, device="cuda")
    sfa = torch.full((G, K // 128, max_m), -3.0, device="cuda")
    dg.dg_m_grouped_scatter_fp8_masked(x.cuda(), None if w is None else dev(w), row_of, slot_of, a, sfa, pow2_scales=pow2)
    torch.cuda.synchronize()
    want_m, want_row, want_slot = around.layout_masked(ids, 0, G, max_m)
    assert np.array_equal(slot_of.cpu().numpy(), want_slot) and np.array_equal(row_of.cpu().numpy(), want_row)
    assert np.array_equal(masked_m.cpu().numpy(), want_m) and want_m[7] == max_m
    codes = a.cpu().numpy().reshape(G * max_m, K)
    sf = sfa.cpu().numpy().transpose(0, 2, 1).reshape(G * max_m, K // 128).astype(np.float64)
    slot = want_slot.ravel()
    assert np.all(codes[slot < 0] == KEEP) and np.all(sf[slot < 0] == -3.0)
    rows = np.nonzero(slot >= 0)[0]
    v = x.double().numpy()[slot[rows] // k]
    if weighted:
        v = v * w.astype(np.float64).ravel()[slot[rows], None]
    v = v.reshape(rows.size, K // 128, 128)
    amax = np.abs(v).max(axis=2)
    if pow2:                     # the power is chosen from the fp32 quotient
        amax = (amax / 448.0).astype(np.float32).astype(np.float64) * 448.0
    check_block_codes(codes[rows].reshape(v.shape), sf[rows][:, :, None], v, amax[:, :, None], pow2)


@pytest.mark.parametrize("ws", [0, 4096, 1 << 20])
def test_masked_layout_with_a_bound_workspace(dg, ws):
    print(f"case: masked layout on a stream with a workspace of {256 + ws} bytes", flush=True)
    rng = np.random.default_rng(14)
    T, k, G, max_m = 9000, 4, 64, 500
    ids = np.stack([rng.permutation(G)[:k] for _ in range(T)]).astype(np.int32)
    st = torch.cuda.Stream()
    buf = torch.zeros(256 + ws, dtype=torch.uint8, device="cuda")
    dg.dg_bind_stream_workspace(st, buf)
    try:
        out = i32(G), i32(T, k), i32(G, max_m)
        d = dev(ids)
        torch.cuda.synchronize()
        dg.dg_m_grouped_layout_masked(d, 0, *out, stream=st)
        st.synchronize()
    finally:
        dg.dg_bind_stream_workspace(st, None)
    for g, r in zip(out, around.layout_masked(ids, 0, G, max_m)):
        assert np.array_equal(g.cpu().numpy(), r)


def test_masked_layouts_on_two_streams(dg):
    # more than 8192 choices: the counts go through each stream's own workspace
    print("case: masked layouts on two streams at once", flush=True)
    rng = np.random.default_rng(15)
    T, k, G, max_m = 20000, 4, 96, 1200
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ids = [rng.integers(0, G, (T, k)).astype(np.int32) for _ in range(2)]
    d_ids = [dev(v) for v in ids]
    outs = [(i32(G), i32(T, k), i32(G, max_m)) for _ in range(2)]
    torch.cuda.synchronize()
    try:
        for s, b in zip(streams, spaces):
            dg.dg_bind_stream_workspace(s, b)
        for _ in range(10):
            for s, v, o in zip(streams, d_ids, outs):
                dg.dg_m_grouped_layout_masked(v, 0, *o, stream=s)
        torch.cuda.synchronize()
    finally:
        for s in streams:
            dg.dg_bind_stream_workspace(s, None)
    for v, o in zip(ids, outs):
        for g, r in zip(o, around.layout_masked(v, 0, G, max_m)):
            assert np.array_equal(g.cpu().numpy(), r)


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
