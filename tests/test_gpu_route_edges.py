"""The router at the ends of fp32: scores below its normal range, large logits in
the sigmoid's gradient, keys of +inf and group scores beyond the largest finite
value.  Each case runs on both kernels (sixteen lanes or a wave per token)."""
import numpy as np
import pytest
import torch

from oracle import around
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

# experts, choices: the second kernel serves more than 512 experts or 16 choices
PATHS = [(64, 4), (200, 12), (512, 16), (640, 4), (48, 20)]


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def backward(dg, x, ids, g, **kw):
    lx = dev(x)
    out = torch.full_like(lx, float("nan"))
    dg.dg_route_topk_backward(lx, dev(ids.astype(np.int32)), dev(g), out, **kw)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", PATHS)
def test_sigmoid_gradient_keeps_its_digits_at_large_logits(dg, E, k, renorm):
    print(f"case: sigmoid gradient at large logits E={E} top_k={k} renormalize={renorm}", flush=True)
    rng = np.random.default_rng(E + k)
    T, scale = 24, 1.5
    x = (rng.uniform(5.0, 40.0, (T, E)) * np.where(rng.random((T, 1)) < 0.8, 1.0, -1.0)).astype(np.float32)
    ids, _, _ = around.route(x, None, k, "sigmoid")
    g = rng.standard_normal((T, k)).astype(np.float32)
    got = backward(dg, x, ids, g, score="sigmoid", renormalize=renorm, scale=scale)
    ref = around.route_backward(x, ids, g, "sigmoid", renorm, scale)
    xs = np.take_along_axis(x, ids, axis=1).astype(np.float64)
    s, rest = 1.0 / (1.0 + np.exp(-xs)), 1.0 / (1.0 + np.exp(xs))
    if renorm:       # u_j = share_j (g_j - sum_i share_i g_i)
        share = s / s.sum(axis=1, keepdims=True)
        size = share * (np.abs(g) + (share * np.abs(g)).sum(axis=1, keepdims=True))
    else:
        size = s * np.abs(g)
    # the oracle's 1 - s cancels in 64 bits too: worked out here from the complement
    u = g * s if not renorm else share * (g - (share * g).sum(axis=1, keepdims=True))
    want = np.zeros_like(ref)
    np.put_along_axis(want, ids, scale * u * rest, axis=1)
    assert np.allclose(want, ref, rtol=1e-6, atol=1e-12)
    # score and complement within 5e-7 each, the sum over at most 20 choices and a few products 2^-24 each
    bound = np.zeros_like(ref)
    np.put_along_axis(bound, ids, 5e-6 * scale * size * rest, axis=1)
    assert np.all(np.abs(got - want) <= bound)
