"""The norm of many gradients and their clipping against fp64.

Bounds: squares and sums are fp64, so the norm is off by its rounding to fp32
(2^-24) and less than 1e-9 besides; the factor has two more fp32 roundings, the
result one of its type."""
import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def tensors(seed, sizes, kinds, scale=1.0):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32)).to(kinds[i % len(kinds)]).cuda()
            for i, n in enumerate(sizes)]


def norm_of(dg, grads):
    norm = torch.full((1,), float("nan"), device="cuda")
    dg.dg_grad_norm(grads, norm)
    torch.cuda.synchronize()
    return norm


def wanted(grads):
    return layer.grad_norm([g.double().cpu().numpy() for g in grads])


F, H = torch.float32, torch.bfloat16
CASES = [
    ([1], [F]), ([1], [H]), ([0, 3, 0], [F]), ([5, 9, 2], [F, H]), ([4096, 17, 70001], [H, F]),
    ([8193, 8192, 8191, 16384, 16385], [F]), ([16385, 16384, 16383, 32769], [H]), ([1000003], [F]), ([2000001], [H]),
    (list(range(1, 260)), [F, H]), ([7] * 500, [H]), ([1 << 22, 3, 1 << 20], [F, H]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{len(c[1])}")
def test_norm_and_clip(dg, case):
    sizes, kinds = case
    print(f"case: grads {len(sizes)} tensors up to {max(sizes)}", flush=True)
    grads = tensors(sum(sizes), sizes, kinds)
    norm = norm_of(dg, grads)
    want = wanted(grads)
    assert abs(float(norm) - want) <= (UNIT + 1e-9) * want
    for max_norm in (0.5 * want, 2.0 * want, 0.0):
        factor = layer.grad_factor(float(norm), float(np.float32(max_norm)))
        outs = [torch.full_like(g, float("nan")) for g in grads]
        dg.dg_grad_clip(grads, outs, norm, max_norm)
        torch.cuda.synchronize()
        for g, o in zip(grads, outs):
            ref = g.double() * factor
            assert ((o.double() - ref).abs() <= (HALF[g.dtype] + 3 * UNIT) * ref.abs() + 1e-38).all()
        if factor == 1.0:
            assert all(torch.equal(g, o) for g, o in zip(grads, outs))
        same = [g.clone() for g in grads]
        dg.dg_grad_clip(same, same, norm, max_norm)
        assert all(torch.equal(o, s) for o, s in zip(outs, same))


def test_views_at_any_element(dg):
    """Tensors of a flat buffer, one behind the other, from odd elements on; what lies between them stays."""
    for kind in (F, H):
        flat = torch.randn(40000, device="cuda").to(kind)
        views = [flat[1:1000], flat[1003:1004], flat[2001:20000], flat[20001:39999]]
        before = flat.clone()
        norm = norm_of(dg, views)
        want = wanted(views)
        assert abs(float(norm) - want) <= (UNIT + 1e-9) * want
        other = torch.zeros(40011, device="cuda", dtype=kind)
        outs = [other[5:1004], other[1004:1005], other[1010:19009], other[20013:40011]]
        dg.dg_grad_clip(views, outs, norm, 1.0)
        dg.dg_grad_clip(views, views, norm, 1.0)
        assert all(torch.equal(a, b) for a, b in zip(views, outs))
        assert torch.equal(flat[[0, 1000, 1001, 1002, 1004, 20000, 39999]], before[[0, 1000, 1001, 1002, 1004, 20000, 39999]])
        assert (other[:5] == 0).all() and (other[1005:1010] == 0).all() and (other[19009:20013] == 0).all()


def test_values_whose_squares_leave_fp32(dg):
    for v in (1e30, 3e-38, 1e-42):
        g = torch.full((1000,), v, device="cuda")
        want = wanted([g])
        assert abs(float(norm_of(dg, [g])) - want) <= (UNIT + 1e-9) * want + 1e-45
    g = torch.full((4,), 3.0e38, device="cuda")
    assert float(norm_of(dg, [g])) == float("inf")


def test_infinities_and_nan(dg):
    g = torch.ones(100, device="cuda")
    g[7] = float("inf")
    norm = norm_of(dg, [g])
    assert float(norm) == float("inf")
    out = torch.empty_like(g)
    dg.dg_grad_clip([g], [out], norm, 1.0)
    assert torch.isnan(out[7]) and (out[:7] == 0).all()
    g[9] = float("nan")
    norm = norm_of(dg, [g])
    assert torch.isnan(norm).all()
    dg.dg_grad_clip([g], [out], norm, 1.0)
    assert torch.isnan(out).all()


def test_no_tensors(dg):
    assert float(norm_of(dg, [])) == 0.0
    norm = torch.ones(1, device="cuda")
    dg.dg_grad_clip([], [], norm, 1.0)
    empty = torch.empty(0, device="cuda")
    assert float(norm_of(dg, [empty])) == 0.0


def test_lists_of_all_kinds(dg):
    """Tuples, generators, parameters and views, through both sides of the binding, give the same bits."""
    grads = tensors(3, [100, 7, 5000], [F, H])
    want = norm_of(dg, grads)
    for same in (tuple(grads), iter(grads), [torch.nn.Parameter(g) for g in grads], [g.view(-1, 1) for g in grads]):
        assert torch.equal(norm_of(dg, same), want)
    other = torch.cuda.Stream()                  # (a stream object takes the checks in Python)
    other.wait_stream(torch.cuda.current_stream())
    norm, outs = torch.empty(1, device="cuda"), [torch.empty_like(g) for g in grads]
    dg.dg_grad_norm(grads, norm, stream=other)
    dg.dg_grad_clip(grads, outs, norm, 1.0, stream=other)
    other.synchronize()
    assert torch.equal(norm, want)
    dg.dg_grad_clip(iter(grads), tuple(grads), want, 1.0)
    assert all(torch.equal(g, o) for g, o in zip(grads, outs))


def test_small_workspace_and_the_same_bits(dg):
    grads = tensors(4, [70000, 3, 900] * 100, [F, H])
    want = norm_of(dg, grads)
    assert torch.equal(want, norm_of(dg, grads))
    stream = torch.cuda.Stream()
    ws = torch.zeros(256 + 24, dtype=torch.uint8, device="cuda")
    dg.dg_bind_stream_workspace(stream, ws)
    try:
        with torch.cuda.stream(stream):
            got = norm_of(dg, grads)
            ref = wanted(grads)
            assert abs(float(got) - ref) <= (UNIT + 1e-9) * ref
    finally:
        dg.dg_bind_stream_workspace(stream, None)
