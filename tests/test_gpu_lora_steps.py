"""Low-rank adapters in the forms that take several column steps per workgroup or
64 columns per wave, and how many bits the inner product keeps."""
import numpy as np
import pytest
import torch

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


def reference(x, a, b, s, ids, c):
    """(result, adapter term's sum of magnitudes) in fp64, adapter by adapter."""
    out = np.zeros((x.shape[0], b.shape[1])) if c is None else c.double().numpy().copy()
    mag = np.zeros_like(out)
    for i in range(a.shape[0]):
        t = np.nonzero(ids == i)[0]
        if t.size:
            A, B, v = a[i].double().numpy(), b[i].double().numpy(), x[t].double().numpy()
            out[t] += s[i] * ((v @ A.T) @ B.T)
            mag[t] = abs(s[i]) * ((np.abs(v) @ np.abs(A).T) @ np.abs(B).T)
    return out, mag


def run_case(dg, T, L, R, N, K, runs, idle, mode, seed):
    rng = np.random.default_rng(seed)
    x, a, b = bf16(rng, T, K), bf16(rng, L, R, K, scale=K ** -0.5), bf16(rng, L, N, R, scale=0.1)
    s = (rng.random(L) + 0.5).astype(np.float32)
    n = -(-T // runs)
    ids = rng.integers(0, L, n)
    ids[rng.random(n) < idle] = -1
    ids = np.repeat(ids, runs)[:T].astype(np.int32)
    c = None if mode == "none" else bf16(rng, T, N)
    d = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    if mode == "in place":
        d.copy_(c)
    cd = None if c is None else d if mode == "in place" else c.cuda()
    dg.dg_lora_bf16_nt(x.cuda(), a.cuda(), b.cuda(), dev(s), dev(ids), cd, d)
    torch.cuda.synchronize()
    ref, mag = reference(x, a, b, s, ids, c)
    got = d.float().cpu().numpy()
    # one rounding to bf16, the inner product's 2^-15 or better, fp32 sums over K and R
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 + (K + R) * 2.0 ** -24) * mag + 1e-37
    err = np.abs(got - ref)
    assert np.all(err <= bound), float((err / bound).max())
    none = ids < 0
    if c is not None:
        assert torch.equal(d.cpu()[torch.from_numpy(none)], c[torch.from_numpy(none)])
    else:
        assert np.all(got[none] == 0.0)


STEPS = [
    # T, adapters, R, N, K, tokens in a row of one adapter, share without one: on 256 CUs a
    # workgroup takes two steps of 64 columns or more
    (4000, 3, 16, 2112, 128, 500, 0.1), (3500, 5, 64, 4096, 256, 333, 0.0), (2500, 2, 128, 2047, 128, 700, 0.1),
    (2000, 3, 256, 4095, 128, 400, 0.2), (6000, 8, 40, 2050, 128, 1, 0.1), (4100, 40, 96, 2500, 128, 1, 0.0),
    (3000, 60, 24, 4100, 128, 1, 0.1), (5000, 300, 32, 2113, 128, 1, 0.0), (3001, 4, 200, 3001, 128, 90, 0.3),
]


@pytest.mark.parametrize("mode", ["none", "c", "in place"])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_several_column_steps_per_workgroup(dg, case, mode):
    T, L, R, N, K, runs, idle = case
    print(f"case: lora steps {case} c={mode}", flush=True)
    tiles = (T + 63 * min(L + 1, T)) // 64
    slots = 4 if R <= 64 else 2 if R <= 128 else 1
    assert (N + 63) // 64 > max(1, slots * 256 // tiles)          # more columns' steps than workgroups for them
    run_case(dg, *case, mode, T + R)


FEW = [
    # up to 256 tokens with four workgroups of 256 columns per CU or more
    (128, 8, 16, 2112, 256, 1, 0.1), (256, 3, 32, 2047, 128, 1, 0.0), (150, 20, 64, 2112, 256, 1, 0.1),
    (200, 7, 128, 1601, 128, 30, 0.2), (256, 2, 256, 1025, 256, 1, 0.0), (255, 100, 24, 4100, 128, 1, 0.3),
    (64, 5, 72, 4099, 384, 1, 0.1), (16, 16, 8, 16387, 128, 1, 0.0),
]


@pytest.mark.parametrize("mode", ["none", "c", "in place"])
@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(map(str, c)))
def test_sixty_four_columns_per_wave(dg, case, mode):
    T, L, R, N, K, runs, idle = case
    print(f"case: lora wide columns {case} c={mode}", flush=True)
    assert T * ((N + 255) // 256) >= 4 * 256
    run_case(dg, *case, mode, T * 3 + R)


@pytest.mark.parametrize("T", [1, 16, 200, 300, 900])
@pytest.mark.parametrize("R", [8, 40, 64, 128, 256])
def test_the_inner_product_keeps_its_fp32_digits(dg, T, R):
    # A x is 1 + 2^-9 + t 2^-20 at rank t and B takes the difference of two ranks: what is left
    # is the last digits, exact in fp32 and in bf16
    print(f"case: lora differences of ranks, {T} tokens of rank {R}", flush=True)
    K, N = 128, 48
    x = torch.ones(T, K, dtype=torch.bfloat16)
    a = torch.zeros(1, R, K)
    a[0, :, 0], a[0, :, 40], a[0, :, 127] = 1.0, 2.0 ** -9, torch.arange(R) * 2.0 ** -20
    b = torch.zeros(1, N, R)
    for n in range(N):
        b[0, n, (3 * n + 1) % R] += 1.0
        b[0, n, (5 * n) % R] -= 1.0
    a, b = a.to(torch.bfloat16), b.to(torch.bfloat16)
    d = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_lora_bf16_nt(x.cuda(), a.cuda(), b.cuda(), None, torch.zeros(T, dtype=torch.int32, device="cuda"), None, d)
    torch.cuda.synchronize()
    ref = ((x.double() @ a[0].double().t()) @ b[0].double().t()).numpy()
    assert np.abs(ref).max() > 0
    assert np.array_equal(d.float().cpu().numpy(), ref)


@pytest.mark.parametrize("T", [3, 300])
def test_an_inner_product_at_the_end_of_fp32(dg, T):
    # beyond bf16's largest value, 3.3895e38, and still an fp32 value; B brings it back
    print(f"case: lora inner product of 3.4e38, {T} tokens", flush=True)
    x = torch.zeros(T, 128, dtype=torch.bfloat16)
    x[:, 0], x[:, 64] = 3.3895e38, 1e36
    x[1], x[2] = -x[1], float("inf")
    a = torch.ones(1, 8, 128, dtype=torch.bfloat16)
    a[0, 1:] = 0.0
    b = torch.zeros(1, 24, 8, dtype=torch.bfloat16)
    b[0, :, 0] = 2.0 ** -100
    d = torch.full((T, 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_lora_bf16_nt(x.cuda(), a.cuda(), b.cuda(), None, torch.zeros(T, dtype=torch.int32, device="cuda"), None, d)
    torch.cuda.synchronize()
    h = x[0].double().sum().item()
    assert 3.397e38 < h < 3.4028e38
    got = d.float().cpu()
    want = torch.full((T, 24), h * 2.0 ** -100)
    want[1] = -want[1]
    keep = [t for t in range(T) if t != 2]                  # an infinity times ranks of 0 is a NaN
    assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs())[keep].all()) and bool(torch.isnan(got[2]).all())
