"""Offsets beyond 2^31 elements and 2^32 bytes in the operands of the balance loss, the
4-bit products and the gradients' clipping, against the fp64 oracle on the rows
concerned."""
import numpy as np
import pytest
import torch

from oracle import layer
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    yield m
    torch.cuda.empty_cache()


def test_balance(dg):
    print("case: balance loss of 2200000 x 1024 logits", flush=True)
    T, E, k = 2200000, 1024, 2
    logits = torch.zeros(T, E, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(0)
    tail = rng.standard_normal((40, E)).astype(np.float32)
    logits[T - 40:] = dev(tail)
    choice = np.argsort(rng.random((40, E)), axis=1)[:, :k].astype(np.int32)
    ids[T - 40:] = dev(choice)
    starts = torch.tensor([0, T - 40, T], dtype=torch.int32, device="cuda")
    loss, counts = torch.empty(2, device="cuda"), torch.empty(2, E, dtype=torch.int32, device="cuda")
    dg.dg_route_balance(logits, ids, starts, loss, counts)
    torch.cuda.synchronize()
    want, n = layer.balance(tail, choice, None, "softmax")
    assert np.array_equal(counts[1].cpu().numpy(), n[0]) and int(counts[0, 0]) == (T - 40) * k
    assert abs(float(loss[1]) - want[0]) <= (E + 160) * 2.0 ** -24 * want[0]
    assert abs(float(loss[0]) - 1.0) < 1e-4                       # equal shares
    out = torch.empty_like(logits)
    dg.dg_route_balance_backward(logits, counts, starts, None, None, out, k)
    torch.cuda.synchronize()
    ref, mag = layer.balance_backward(tail, n, None, None, None, k, "softmax")
    got = out[T - 40:].double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + (E + 33) * 2.0 ** -24 * mag + 1e-37)


def test_experts(dg):
    print("case: 4-bit products with 330 experts of 4096 x 7168", flush=True)
    rng = np.random.default_rng(1)
    G, N, K = 330, 4096, 7168                                     # 4.8 GB of codes
    b = torch.zeros(G, N, K // 2, dtype=torch.uint8, device="cuda")
    far = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    b[G - 1] = dev(far)
    sfb = torch.full((G, K // 128, N), 0x7C7C7C7C, dtype=torch.int32, device="cuda")
    x = torch.from_numpy(rng.standard_normal((3, K)).astype(np.float32)).to(torch.bfloat16)
    ids = torch.tensor([[G - 1, 0], [5, G - 1], [1, 2]], dtype=torch.int32, device="cuda")
    d = torch.full((6, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x.cuda(), ids, 0, b, sfb, None, d)
    torch.cuda.synchronize()
    w = layer.fp4_weights(far, np.full((K // 128, N), 0x7C7C7C7C, dtype=np.int32))
    ref, mag = layer.gemv(x.double().numpy()[:2], w, None)
    got = d.double().cpu().numpy()
    assert np.all(np.abs(got[[0, 3]] - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * K * 2.0 ** -23 * mag)
    assert np.all(got[[1, 2, 4, 5]] == 0)


def test_rows_far_apart(dg):
    print("case: 4-bit products with rows of x and d 2^30 elements apart", flush=True)
    rng = np.random.default_rng(2)
    N, K, far = 40, 256, 1 << 30
    x = torch.zeros(2 * far + K, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(2 * far + N, dtype=torch.bfloat16, device="cuda")
    v = torch.from_numpy(rng.standard_normal((3, K)).astype(np.float32)).to(torch.bfloat16)
    xs, ds = torch.as_strided(x, (3, K), (far, 1)), torch.as_strided(d, (3, N), (far, 1))
    xs.copy_(v)
    b = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = rng.random((K // 32, N)).astype(np.float32)
    dg.dg_bf16_int4_gemv_nt(xs, dev(b), dev(s), None, None, ds)
    torch.cuda.synchronize()
    w, most = layer.int4_weights(b, s, None)
    ref, mag = layer.gemv(v.double().numpy(), w, None, most)
    assert np.all(np.abs(ds.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * K * 2.0 ** -23 * mag)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients(dg, dtype):
    print("case: a gradient of 2^31 + 5 elements", flush=True)
    n = (1 << 31) + 5
    g = torch.zeros(n, dtype=dtype, device="cuda")
    g[-3:] = torch.tensor([3.0, -4.0, 12.0], dtype=dtype, device="cuda")
    norm = torch.empty(1, device="cuda")
    dg.dg_grad_norm([g], norm)
    assert float(norm) == 13.0
    dg.dg_grad_clip([g], [g], norm, 6.5)
    torch.cuda.synchronize()
    f = 6.5 / (13.0 + 1e-6)
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    ref = torch.tensor([3.0, -4.0, 12.0], dtype=torch.double) * f
    assert ((g[-3:].double().cpu() - ref).abs() <= (half + 3 * 2.0 ** -24) * ref.abs()).all()
    assert int(torch.count_nonzero(g[:1 << 30])) == 0 and int(torch.count_nonzero(g[1 << 30:-3])) == 0
