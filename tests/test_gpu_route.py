"""The router and its gradient against the fp64 oracle: choices exactly (ties to
the lowest index, rows drawn clear of 32-bit near-ties otherwise), weights and
gradients within bounds derived from fp32 rounding."""
import numpy as np
import pytest
import torch

from oracle import around
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

# Weights: x - top rounds to 2^-24 |x - top| (|x - top| <= 32 here: 2e-6 in the
# exponent), the exponential, the sum of up to 1024 terms and the divisions a
# few 1e-7 each.
W_RTOL = 5e-6
# Gradients: sums of at most 64 such terms of size max|grad| * scale.
G_RTOL = 1e-5


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def draw(rng, T, E, bf16, top_k, score, bias, masked=0.0, **kw):
    """Logits whose choices do not hang on 32-bit rounding."""
    def fresh(n):
        x = (rng.standard_normal((n, E)) * 1.5).astype(np.float32)
        if bf16:
            x = (x.view(np.uint32) & 0xFFFF0000).view(np.float32)
        if masked:
            x[rng.random((n, E)) < masked] = -np.inf
        return x
    x = fresh(T)
    for _ in range(50):
        ids, w, margin = around.route(x, bias, top_k, score, **kw)
        # equal logits tie exactly where there is no bias, and are not redrawn
        bad = np.nonzero((margin < 1e-5) & ((margin > 0) | (bias is not None) | (kw.get("num_groups", 1) > 1)))[0]
        if bad.size == 0:
            return x, ids, w
        x[bad] = fresh(bad.size)
    raise AssertionError("no clear inputs found")


def run(dg, x, bias, top_k, bf16=False, **kw):
    T = x.shape[0]
    lx = dev(x).to(torch.bfloat16) if bf16 else dev(x)
    ids = torch.full((T, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, top_k), float("nan"), device="cuda")
    dg.dg_route_topk(lx, None if bias is None else dev(bias), ids, w, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


CASES = [
    # T, E, top_k, score, groups, kept, group_top, bias, bf16, renormalize, scale, masked
    (1, 1, 1, "softmax", 1, 1, 1, False, False, True, 1.0, 0.0),
    (1, 256, 8, "sigmoid", 8, 4, 2, True, False, True, 2.5, 0.0),
    (67, 256, 8, "sigmoid", 8, 4, 2, True, False, True, 2.5, 0.0),
    (130, 256, 8, "sigmoid", 8, 4, 2, True, True, False, 1.0, 0.03),
    (5, 8, 2, "softmax", 1, 1, 1, False, False, True, 1.0, 0.0),
    (33, 60, 4, "softmax", 1, 1, 1, False, True, True, 1.0, 0.1),
    (9, 63, 6, "softmax", 3, 2, 1, False, False, False, 16.0, 0.0),
    (17, 160, 6, "softmax", 8, 3, 1, True, False, True, 1.0, 0.0),
    (4, 65, 64, "softmax", 1, 1, 1, False, False, True, 1.0, 0.0),
    (3, 512, 10, "sigmoid", 64, 20, 2, False, False, True, 1.0, 0.0),
    (6, 1024, 16, "softmax", 1, 1, 1, True, False, True, 1.0, 0.0),
    (5, 1000, 33, "sigmoid", 4, 4, 2, True, True, False, 1.0, 0.2),
    (11, 48, 48, "sigmoid", 1, 1, 1, False, False, True, 1.0, 0.3),
    (7, 16, 4, "sigmoid", 16, 5, 2, True, False, True, 1.0, 0.0),
    (13, 384, 9, "softmax", 16, 7, 2, False, False, True, 1.0, 0.5),
    (1023, 128, 1, "sigmoid", 1, 1, 1, True, False, False, 1.0, 0.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_choice_and_weights(dg, case):
    T, E, k, score, G, kept, gt, with_bias, bf16, renorm, scale, masked = case
    print(f"case: route {case}", flush=True)
    rng = np.random.default_rng(E * 7 + T)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
    kw = dict(num_groups=G, topk_groups=kept, group_top=gt, renormalize=renorm, scale=scale)
    x, ids, w = draw(rng, T, E, bf16, k, score, bias, masked=masked, **kw)
    got_ids, got_w = run(dg, x, bias, k, bf16, score=score, **kw)
    assert np.array_equal(got_ids, ids)
    assert np.all(np.abs(got_w - w) <= W_RTOL * np.abs(w) + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,kept", [(40, 1, 1), (64, 8, 3), (256, 8, 4), (300, 10, 4), (1024, 32, 5)])
def test_ties_go_to_the_lowest_index(dg, score, E, G, kept):
    # few distinct logits: every choice is made among equals
    print(f"case: route ties {score} E={E} groups={G}", flush=True)
    rng = np.random.default_rng(E)
    x = rng.integers(0, 3, (37, E)).astype(np.float32)
    x[0] = 0.0
    for group_top in (1, 2):
        kw = dict(num_groups=G, topk_groups=kept, group_top=group_top)
        ids, w, _ = around.route(x, None, 12, score, **kw)
        got_ids, got_w = run(dg, x, None, 12, score=score, **kw)
        assert np.array_equal(got_ids, ids)
        assert np.all(np.abs(got_w - w) <= W_RTOL * np.abs(w))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(8, 1), (96, 4), (320, 8)])
def test_masked_experts_and_rows_of_extremes(dg, score, E, G):
    print(f"case: route extremes {score} E={E} groups={G}", flush=True)
    lowest = np.finfo(np.float32).min
    x = np.tile(np.linspace(-1.0, 1.0, E, dtype=np.float32), (10, 1))
    x[0] = -np.inf                                  # nothing left
    x[1] = np.nan
    x[2, 1:] = -np.inf                              # one left
    x[3, :] = lowest                                # the type's lowest value is no mask
    x[4, 3] = np.inf
    x[5, ::2] = np.nan
    x[6, :] = -200.0                                # sigmoid scores underflow to 0
    x[7, E // G:] = -np.inf                         # one group left
    x[8, 0], x[8, 1] = np.inf, np.inf
    x[9, :] = 100.0
    bias = np.zeros(E, dtype=np.float32)
    bias[2], bias[5] = -np.inf, np.nan              # a bias masks too
    k = min(6, E // G * max(1, G // 2))
    for b in (None, bias):
        for renorm in (True, False):
            kw = dict(num_groups=G, topk_groups=max(1, G // 2), group_top=2, renormalize=renorm, scale=1.5)
            ids, w, margin = around.route(x, b, k, score, **kw)
            got_ids, got_w = run(dg, x, b, k, score=score, **kw)
            # -200's sigmoid is 1.4e-87 in 64 bits and 0 in 32: ties, and weights of zero
            rows = [t for t in range(10) if not (score == "sigmoid" and t in (3, 6))]
            assert np.array_equal(got_ids[rows], ids[rows])
            assert np.all(np.abs(got_w - w)[rows] <= W_RTOL * np.abs(w[rows]) + 1e-37)
            if score == "sigmoid":
                free = [e for e in range(E // G * max(1, G // 2)) if b is None or e not in (2, 5)]
                for t in (3, 6):
                    assert list(got_ids[t]) == (free + [-1] * k)[:k] and np.all(got_w[t] == 0.0)


@pytest.mark.parametrize("case", [c for c in CASES if c[0] < 500], ids=lambda c: "-".join(map(str, c)))
def test_gradient(dg, case):
    T, E, k, score, G, kept, gt, with_bias, bf16, renorm, scale, masked = case
    print(f"case: route gradient {case}", flush=True)
    rng = np.random.default_rng(E * 11 + T)
    x = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    if bf16:
        x = (x.view(np.uint32) & 0xFFFF0000).view(np.float32)
    if masked:
        x[rng.random((T, E)) < masked] = -np.inf
    ids, _, _ = around.route(x, None, k, score)
    ids = ids.astype(np.int32)
    if T > 2:
        ids[1, -1], ids[2, 0] = -1, E + 3           # slots that take no part
        ids[0] = rng.permutation(E)[:k]             # any choice, masked experts too
    g = rng.standard_normal((T, k)).astype(np.float32)
    g[ids < 0] = np.nan                             # what stands in an empty slot is not read
    ref = around.route_backward(x, ids, np.where(np.isnan(g), 0.0, g), score, renorm, scale)
    lx = dev(x).to(torch.bfloat16) if bf16 else dev(x)
    out = torch.full_like(lx, float("nan"))
    dg.dg_route_topk_backward(lx, dev(ids), dev(g), out, score=score, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy().astype(np.float64)
    most = np.nanmax(np.abs(g), axis=1, keepdims=True) * scale if k else 0.0
    bound = G_RTOL * most + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(dg, score, renorm):
    print(f"case: route gradient by differences {score} renormalize={renorm}", flush=True)
    rng = np.random.default_rng(5)
    T, E, k, scale = 3, 20, 4, 2.0
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids, _, _ = around.route(x, None, k, score)
    g = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.empty(T, E, device="cuda")
    dg.dg_route_topk_backward(dev(x), dev(ids.astype(np.int32)), dev(g), out, score=score, renormalize=renorm,
                              scale=scale)
    torch.cuda.synchronize()
    h = 1e-5                                        # central differences of the fp64 definition: error h^2 and 1e-16 / h
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        up = around.route_weights(x + d, ids, score, renorm, scale)
        down = around.route_weights(x - d, ids, score, renorm, scale)
        ref = ((up - down) / (2 * h) * g).sum(axis=1)
        assert np.all(np.abs(out[:, e].cpu().numpy() - ref) <= G_RTOL * np.abs(g).max() * scale)
