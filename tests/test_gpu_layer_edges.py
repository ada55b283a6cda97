"""Balance loss, 4-bit products and gradients' calls at sizes and values that dg.h allows
and that no step of a model has."""
import numpy as np
import pytest
import torch

from oracle import layer
from tests.exact4 import decode, draw, generator, product, quarters, whole
from tests.gpu_util import dev
from tests.test_gpu_balance import UNIT, forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    yield m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,S", [(1000, 1 << 20), (1000, (1 << 20) + 1), (60000, 1100000)])
def test_more_sequences_than_a_launch_has(dg, T, S):
    """Most of them empty; the loss and the gradient of the others."""
    print(f"case: balance of {T} tokens in {S} sequences", flush=True)
    E, k = 4, 2
    rng = np.random.default_rng(S)
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    starts = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    loss, counts = forward(dg, torch.from_numpy(x), ids, starts, "softmax")
    p, _ = layer.shares(x, "softmax")
    seq = np.searchsorted(starts[1:], np.arange(T), side="right")             # the first that ends behind the token
    inside = (seq < S) & (np.arange(T) >= starts[0])
    n = np.zeros((S, E))
    sums = np.zeros((S, E))
    for j in range(k):
        np.add.at(n, (seq[inside], ids[inside, j]), 1)
    np.add.at(sums, seq[inside], p[inside])
    length = np.diff(starts).astype(np.float64)
    want = np.divide(E * (n * sums).sum(1), k * length ** 2, out=np.zeros(S), where=length > 0)
    assert np.array_equal(counts, n)
    assert np.all(np.abs(loss - want) <= (E + 160) * UNIT * want)
    grad_loss = rng.standard_normal(S).astype(np.float32)
    out = torch.empty(T, E, device="cuda")
    dg.dg_route_balance_backward(torch.from_numpy(x).cuda(), dev(n.astype(np.int32)), dev(starts), dev(grad_loss), None, out, k)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    at = np.clip(seq, 0, S - 1)
    w = np.where(inside, E / (k * length[at].clip(1) ** 2) * grad_loss[at], 0.0)[:, None]
    f = n[at]
    g = w * p * (f - (p * f).sum(1, keepdims=True))
    mag = np.abs(w) * p * (np.abs(f) + (p * np.abs(f)).sum(1, keepdims=True)) * 2
    assert np.all(np.abs(got - g) <= UNIT * np.abs(g) + (E + 33) * UNIT * mag + 1e-37)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 7, 20])
def test_zero_points_beyond_the_integers_and_negative_scales(dg, group, M):
    """Zero points of 0 to 255, scales of either sign: sums of at most 2176 * 2 * 270 * 2 halves, exact in fp32."""
    print(f"case: int4 with zero points up to 255, groups of {group}, {M} tokens", flush=True)
    g = generator(group + M)
    N, K = 130, 2176
    b, z = draw(g, 0, 256, N, K // 2), draw(g, 0, 256, K // group, N)
    s = torch.exp2(draw(g, -1, 2, K // group, N, dtype=torch.int8).float()) * (draw(g, 0, 2, K // group, N) * 2.0 - 1.0)
    x, c = whole(g, M, K), quarters(g, M, N)
    d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_int4_gemv_nt(x, b, s, z, c, d)
    torch.cuda.synchronize()
    assert torch.equal(d, product(x, decode(("int4", group), b, s, z), c))


def test_tensors_without_dimensions(dg):
    grads = [torch.tensor(3.0, device="cuda"), torch.tensor(-4.0, device="cuda", dtype=torch.bfloat16),
             torch.full((1, 1, 1), 12.0, device="cuda")]
    norm = torch.empty(1, device="cuda")
    dg.dg_grad_norm(grads, norm)
    assert float(norm) == 13.0
    dg.dg_grad_clip(grads, grads, norm, 13.0 + 1e-6)
    assert [float(t) for t in grads] == [3.0, -4.0, 12.0]
    dg.dg_grad_clip(grads, grads, norm, 0.0)
    assert [float(t) for t in grads] == [0.0, 0.0, 0.0]


def test_many_launches_of_tensors(dg):
    """5003 tensors of 0 to 40 values: 42 launches, in one list, clipped out of place and in place."""
    print("case: 5003 gradients", flush=True)
    rng = np.random.default_rng(0)
    sizes = rng.integers(0, 41, 5003)
    flat = [torch.randn(int(sizes.sum()), device="cuda").to(t) for t in (torch.float32, torch.bfloat16)]
    parts = [f.split(sizes.tolist()) for f in flat]
    grads = [parts[i % 2][i] for i in range(len(sizes))]
    norm = torch.empty(1, device="cuda")
    dg.dg_grad_norm(grads, norm)
    want = torch.cat([g.double() for g in grads]).square().sum().sqrt()
    assert abs(float(norm) - float(want)) <= (2.0 ** -24 + 1e-9) * float(want)
    outs = [torch.full_like(g, float("nan")) for g in grads]
    dg.dg_grad_clip(grads, outs, norm, 1.0)
    torch.cuda.synchronize()
    f = 1.0 / (float(norm) + 1e-6)
    for kind, half in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        g = torch.cat([t for t in grads if t.dtype == kind]).double() * f
        o = torch.cat([t for t in outs if t.dtype == kind]).double()
        assert bool(((o - g).abs() <= (half + 3 * 2.0 ** -24) * g.abs() + 1e-38).all())
    others = [parts[1 - i % 2][i].clone() for i in range(len(sizes))]
    dg.dg_grad_clip(grads, grads, norm, 1.0)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    assert all(torch.equal(parts[1 - i % 2][i], others[i]) for i in range(len(sizes)))
