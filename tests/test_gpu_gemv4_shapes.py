"""The 4-bit products on every launch shape (columns per workgroup, waves, tokens per
tile) at odd numbers of 128-K blocks, on choices that repeat an expert, and by lists.
Bounds as in test_gpu_gemv4.py; the fp64 reference is multiplied on the GPU."""
import numpy as np
import pytest
import torch

from oracle import layer
from tests.gpu_util import dev
from tests.test_gpu_gemv4 import FORMS, bf16, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def check(d, x, w, most, c, K):
    x, w, most = x.double().cuda(), dev(w), dev(most)
    ref, mag = x @ w.t(), x.abs() @ most.t()
    if c is not None:
        ref, mag = ref + c.double().cuda(), mag + c.double().abs().cuda()
    bound = 2.0 ** -8 * ref.abs() + (K + K // 16 + 16) * 2.0 ** -23 * mag + 1e-37
    assert bool(((d.double() - ref).abs() <= bound).all()), float(((d.double() - ref).abs() / bound).max())


# one workgroup per CU or more with 64, 32 or 16 columns each, or fewer, at 256 CUs
SHAPES = [
    (64, 4200, 384), (20, 8300, 640), (64, 2112, 384), (18, 4100, 640), (17, 2112, 384), (24, 100, 1152),
    (8, 8300, 384), (7, 4200, 640), (6, 500, 1152),
    (3, 8300, 4224), (4, 8300, 640), (1, 8300, 384), (2, 4200, 1152), (4, 77, 2176), (1, 4097, 128),
]


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("size", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_launch_shapes(dg, size, form):
    M, N, K = size
    print(f"case: gemv shape {size} {form}", flush=True)
    rng = np.random.default_rng(M * 7 + N + K)
    args, w, most = weights(rng, form, (), N, K)
    x, c = bf16(rng, M, K), bf16(rng, M, N)
    d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    call = dg.dg_bf16_fp4_gemv_nt if form == "fp4" else dg.dg_bf16_int4_gemv_nt
    call(x.cuda(), *args, c.cuda(), d)
    torch.cuda.synchronize()
    check(d, x, w[0], most[0], c, K)


REPEATED = [
    # T, top_k, experts, N, K: every id drawn on its own, so that tokens repeat an expert
    (1, 40, 2, 130, 384), (3, 9, 1, 70, 256), (4, 300, 3, 40, 128), (6, 20, 2, 100, 640), (8, 250, 5, 33, 128),
    (2, 1500, 4, 24, 128), (7, 400, 3, 40, 256), (64, 3, 1, 65, 384), (700, 4, 2, 20, 128), (1, 1, 1, 4300, 384),
    (30, 8, 4, 8300, 128), (64, 8, 300, 2112, 128),
]


@pytest.mark.parametrize("form", FORMS[:3], ids=str)
@pytest.mark.parametrize("case", REPEATED, ids=lambda s: "-".join(map(str, s)))
def test_repeated_experts(dg, case, form):
    T, k, G, N, K = case
    print(f"case: gemv by repeated choices {case} {form}", flush=True)
    rng = np.random.default_rng(T + k + N)
    args, w, most = weights(rng, form, (G,), N, K)
    ids = rng.integers(-1, G + 1, (T, k)).astype(np.int32)
    x = bf16(rng, T, K)
    d = torch.full((T * k, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    call = dg.dg_m_grouped_bf16_fp4_gemv_nt_topk if form == "fp4" else dg.dg_m_grouped_bf16_int4_gemv_nt_topk
    call(x.cuda(), dev(ids), 0, *args, None, d)
    torch.cuda.synchronize()
    flat, row = ids.ravel(), np.repeat(np.arange(T), k)
    for e in range(G):
        at = np.nonzero(flat == e)[0]
        if len(at):
            check(d[torch.from_numpy(at).cuda()], x[row[at]], w[e], most[e], None, K)
    assert bool((d[torch.from_numpy(np.nonzero((flat < 0) | (flat >= G))[0]).cuda()] == 0).all())


def test_ids_at_the_ends_of_int32(dg):
    """Ids far from [first, first + G), on both sides, are choices of other experts."""
    rng = np.random.default_rng(0)
    args, w, most = weights(rng, "fp4", (3,), 20, 128)
    ids = np.array([[-2 ** 31, 2 ** 31 - 1, 2 ** 30, 5, 6], [7, 8, -1, 4, 2 ** 31 - 3]], dtype=np.int32)
    x = bf16(rng, 2, 128)
    for T in (2, 900):                                            # counted in place, and by lists
        many = np.concatenate([ids] * (T // 2))
        d = torch.full((T * 5, 20), float("nan"), dtype=torch.bfloat16, device="cuda")
        dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(torch.cat([x] * (T // 2)).cuda(), dev(many), 5, *args, None, d)
        got = d.view(T // 2, 10, 20)
        for place, token, e in ((3, 0, 0), (4, 0, 1), (5, 1, 2)):
            for i in range(T // 2):
                if i in (0, T // 2 - 1):
                    check(got[i, place].view(1, 20), x[token:token + 1], w[e], most[e], None, 128)
        others = [0, 1, 2, 6, 7, 8, 9]
        assert bool((got[:, others] == 0).all())


def test_rows_that_repeat_are_the_same_bits(dg):
    """The same token in any place of any tile gives the same bits."""
    rng = np.random.default_rng(1)
    for form in (FORMS[0], FORMS[3]):
        args, _, _ = weights(rng, form, (2,), 300, 1152)
        x = bf16(rng, 1, 1152).cuda()
        call = dg.dg_m_grouped_bf16_fp4_gemv_nt_topk if form == "fp4" else dg.dg_m_grouped_bf16_int4_gemv_nt_topk
        ids = torch.zeros(90, 1, dtype=torch.int32, device="cuda")
        ids[::7] = 1
        d = torch.empty(90, 300, dtype=torch.bfloat16, device="cuda")
        call(x.expand(90, -1).contiguous(), ids, 0, *args, None, d)
        for e in (0, 1):
            rows = d[(ids == e).view(-1)]
            assert bool((rows == rows[0]).all())


@pytest.mark.parametrize("n", [1, 17, 63, 64, 65, 511, 1023, 1024, 1025, 2047, 2048, 2049])
@pytest.mark.parametrize("G", [1, 3, 1024])
def test_choices_around_the_lists(dg, n, G):
    """One choice per token, with several tiles per expert, ids counted by every workgroup or listed."""
    print(f"case: gemv of {n} choices of {G} experts", flush=True)
    rng = np.random.default_rng(n + G)
    N, K = 20, 128
    args, w, most = weights(rng, "fp4", (G,), N, K)
    ids = rng.integers(-1, G + 1, (n, 1)).astype(np.int32)
    x = bf16(rng, n, K)
    d = torch.full((n, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x.cuda(), dev(ids), 0, *args, None, d)
    torch.cuda.synchronize()
    flat, xd = ids.ravel(), x.double()
    here = (flat >= 0) & (flat < G)
    wd, md = torch.from_numpy(np.asarray(w, dtype=np.float64)), torch.from_numpy(np.asarray(most, dtype=np.float64))
    at = torch.from_numpy(np.clip(flat, 0, G - 1).astype(np.int64))
    ref = torch.empty(n, N, dtype=torch.float64)
    mag = torch.empty(n, N, dtype=torch.float64)
    for i in range(n):
        ref[i], mag[i] = wd[at[i]] @ xd[i], md[at[i]] @ xd[i].abs()
    keep = torch.from_numpy(here)[:, None]
    ref, mag = ref * keep, mag * keep
    bound = 2.0 ** -8 * ref.abs() + (K + K // 16 + 16) * 2.0 ** -23 * mag + 1e-37
    assert bool(((d.cpu().double() - ref).abs() <= bound).all())
