"""Low-rank adapters against the fp64 oracle, with a bound derived from the
stated precision: fp32 sums over K, the inner product kept to 16 bits or more,
one rounding to bf16."""
import numpy as np
import pytest
import torch

from oracle import around
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def check(got, ref, mag, K, R, what=""):
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 + (K + R) * 2.0 ** -24) * mag + 1e-37
    assert np.all(err <= bound), (what, float((err / bound).max()))


def problem(rng, T, L, R, N, K):
    return (bf16(rng, T, K), bf16(rng, L, R, K, scale=K ** -0.5), bf16(rng, L, N, R, scale=0.1),
            (rng.random(L) + 0.5).astype(np.float32))


def assignment(rng, T, L, runs, idle):
    n = -(-T // runs)
    ids = rng.integers(0, L, n)
    ids[rng.random(n) < idle] = -1
    return np.repeat(ids, runs)[:T].astype(np.int32)


CASES = [
    # T, adapters, R, N, K, tokens in a row of one adapter, share without one
    (1, 1, 8, 1, 128, 1, 0.0), (1, 3, 16, 2112, 7168, 1, 0.0), (1, 2, 64, 513, 1024, 1, 0.0),
    (2, 5, 24, 100, 256, 1, 0.0), (15, 4, 16, 129, 384, 1, 0.3), (17, 1, 32, 1000, 640, 1, 0.0),
    (64, 48, 16, 272, 2048, 1, 0.1), (64, 64, 128, 130, 256, 1, 0.0), (63, 2, 8, 96, 512, 1, 0.5),
    (130, 3, 64, 257, 256, 40, 0.1), (257, 300, 16, 64, 128, 1, 0.2), (300, 2, 256, 65, 256, 100, 0.0),
    (1000, 8, 16, 130, 128, 333, 0.0), (513, 1, 40, 31, 128, 600, 0.0), (2049, 7, 8, 33, 128, 1, 0.1),
    (40, 1024, 8, 24, 128, 1, 0.0), (5000, 3, 32, 40, 128, 700, 0.3), (31, 6, 48, 7, 16384, 1, 0.0),
]


@pytest.mark.parametrize("with_c", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_adapters(dg, case, with_c):
    T, L, R, N, K, runs, idle = case
    print(f"case: lora {case} with_c={with_c}", flush=True)
    rng = np.random.default_rng(T * 3 + R + N)
    x, a, b, s = problem(rng, T, L, R, N, K)
    ids = assignment(rng, T, L, runs, idle)
    c = bf16(rng, T, N) if with_c else None
    d = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_lora_bf16_nt(x.cuda(), a.cuda(), b.cuda(), dev(s), dev(ids), None if c is None else c.cuda(), d)
    torch.cuda.synchronize()
    ref, mag = around.lora(x.float().numpy(), a.float().numpy(), b.float().numpy(), s, ids,
                           None if c is None else c.float().numpy())
    check(d.float().cpu().numpy(), ref, mag, K, R)
    none = ids < 0
    if with_c:                                       # without an adapter the projection's bits pass through
        assert torch.equal(d.cpu()[torch.from_numpy(none)], c[torch.from_numpy(none)])
    else:
        assert np.all(d.float().cpu().numpy()[none] == 0.0)


def test_in_place_without_scales_and_ids_out_of_range(dg):
    print("case: lora in place, no scales, ids out of range", flush=True)
    rng = np.random.default_rng(0)
    T, L, R, N, K = 20, 3, 16, 70, 256
    x, a, b, _ = problem(rng, T, L, R, N, K)
    ids = rng.integers(0, L, T).astype(np.int32)
    ids[[0, 5, 9]] = [L, -2**31, 2**31 - 1]
    c = bf16(rng, T, N)
    d = c.cuda()
    dg.dg_lora_bf16_nt(x.cuda(), a.cuda(), b.cuda(), None, dev(ids), d, d)
    torch.cuda.synchronize()
    ref, mag = around.lora(x.float().numpy(), a.float().numpy(), b.float().numpy(), None, ids, c.float().numpy())
    check(d.float().cpu().numpy(), ref, mag, K, R)
    assert torch.equal(d.cpu()[[0, 5, 9]], c[[0, 5, 9]])


@pytest.mark.parametrize("T", [1, 12, 90, 400])
@pytest.mark.parametrize("N,off", [(96, 8), (100, 3), (65, 1)])
def test_column_slices(dg, T, N, off):
    # x, c and d are columns of wider matrices; what lies beside d stays
    print(f"case: lora on column slices T={T} N={N} offset {off}", flush=True)
    rng = np.random.default_rng(T)
    L, R, K = 4, 16, 256
    x, a, b, s = problem(rng, T, L, R, N, K)
    ids = assignment(rng, T, L, 3, 0.2)
    c = bf16(rng, T, N)
    wx = torch.zeros(T, K + 24, dtype=torch.bfloat16, device="cuda")
    wx[:, 8:8 + K] = x.cuda()
    wc = torch.zeros(T, N + 31, dtype=torch.bfloat16, device="cuda")
    wc[:, off:off + N] = c.cuda()
    wd = torch.full((T, N + 17), 7.0, dtype=torch.bfloat16, device="cuda")
    dg.dg_lora_bf16_nt(wx[:, 8:8 + K], a.cuda(), b.cuda(), dev(s), dev(ids), wc[:, off:off + N], wd[:, off:off + N])
    torch.cuda.synchronize()
    ref, mag = around.lora(x.float().numpy(), a.float().numpy(), b.float().numpy(), s, ids, c.float().numpy())
    check(wd[:, off:off + N].float().cpu().numpy(), ref, mag, K, R)
    assert torch.all(wd[:, :off] == 7.0) and torch.all(wd[:, off + N:] == 7.0)


def test_no_adapters_no_rank_no_depth(dg):
    print("case: lora with nothing to add", flush=True)
    rng = np.random.default_rng(1)
    c = bf16(rng, 9, 33)
    ids = torch.zeros(9, dtype=torch.int32, device="cuda")
    for L, R, K in ((0, 16, 128), (2, 0, 128), (2, 16, 0)):
        z = dict(dtype=torch.bfloat16, device="cuda")
        d = torch.full((9, 33), float("nan"), **z)
        dg.dg_lora_bf16_nt(torch.ones(9, K, **z), torch.ones(L, R, K, **z), torch.ones(L, 33, R, **z), None, ids,
                           c.cuda(), d)
        torch.cuda.synchronize()
        assert torch.equal(d.cpu(), c)


def test_rows_without_the_adapter_do_not_see_its_values(dg):
    print("case: lora beside adapters of NaN and infinities", flush=True)
    rng = np.random.default_rng(6)
    x, a, b, s = problem(rng, 40, 3, 16, 50, 256)
    a[1], b[1] = float("nan"), float("inf")
    x[7] = float("nan")
    ids = np.zeros(40, dtype=np.int32)
    ids[20:] = 2
    ids[7] = -1
    ids[11] = 1
    d = torch.empty(40, 50, dtype=torch.bfloat16, device="cuda")
    dg.dg_lora_bf16_nt(x.cuda(), a.cuda(), b.cuda(), dev(s), dev(ids), None, d)
    torch.cuda.synchronize()
    got = d.float().cpu().numpy()
    assert np.isnan(got[11]).all() and np.all(got[7] == 0.0)
    keep = np.array([t for t in range(40) if t != 11])
    ref, mag = around.lora(np.nan_to_num(x.float().numpy()), np.nan_to_num(a.float().numpy()),
                           np.nan_to_num(b.float().numpy(), posinf=0), s, ids, None)
    check(got[keep], ref[keep], mag[keep], 256, 16)


WIDE = [
    # ranks beyond the common ones on both sides of the token count that changes the kernels
    (20, 3, 256, 65, 512, 1, 0.1), (9, 2, 200, 70, 1152, 4, 0.0), (256, 5, 136, 33, 256, 1, 0.1),
    (257, 5, 136, 129, 640, 1, 0.1), (600, 2, 72, 200, 384, 100, 0.2), (1500, 3, 96, 1, 128, 1, 0.0),
    (400, 1024, 16, 20, 256, 1, 0.0), (256, 256, 8, 3, 1024, 1, 0.0), (900, 4, 256, 130, 128, 64, 0.1),
]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)))
def test_ranks_and_token_counts_at_the_kernels_limits(dg, case):
    T, L, R, N, K, runs, idle = case
    print(f"case: lora limits {case}", flush=True)
    rng = np.random.default_rng(T * 5 + R + N)
    x, a, b, s = problem(rng, T, L, R, N, K)
    ids = assignment(rng, T, L, runs, idle)
    c = bf16(rng, T, N)
    d = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_lora_bf16_nt(x.cuda(), a.cuda(), b.cuda(), dev(s), dev(ids), c.cuda(), d)
    torch.cuda.synchronize()
    ref, mag = around.lora(x.float().numpy(), a.float().numpy(), b.float().numpy(), s, ids, c.float().numpy())
    check(d.float().cpu().numpy(), ref, mag, K, R)
