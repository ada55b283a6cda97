"""The router at the ends of fp32: scores below its normal range, large logits in
the sigmoid's gradient, keys of +inf and group scores beyond the largest finite
value.  Each case runs on both kernels (sixteen lanes or a wave per token)."""
import numpy as np
import pytest
import torch

from oracle import around
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -149                                  # fp32's smallest value
MOST = float(np.finfo(np.float32).max)
# experts, choices: the second kernel serves more than 512 experts or 16 choices
PATHS = [(64, 4), (200, 12), (512, 16), (640, 4), (48, 20)]


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def run(dg, x, bias, top_k, **kw):
    T = x.shape[0]
    ids = torch.full((T, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, top_k), float("nan"), device="cuda")
    dg.dg_route_topk(dev(x), None if bias is None else dev(bias), ids, w, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


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


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", PATHS)
def test_scores_below_the_normal_range(dg, score, E, k):
    # e^-88 .. e^-95 are subnormal numbers of fp32, 2^-127 to 2^-137: they order the
    # choice, and their ratios are the weights
    print(f"case: route subnormal scores {score} E={E} top_k={k}", flush=True)
    rng = np.random.default_rng(E * 3 + k)
    T = 18
    x = np.stack([rng.permutation(np.linspace(-95.0, -88.0, E)) for _ in range(T)]).astype(np.float32)
    if score == "softmax":
        x[:, E // 3] = 0.0
    x[-1, ::2] = -np.inf
    for renorm in (True, False):
        ids, w, _ = around.route(x, None, k, score, renormalize=renorm, scale=2.0)
        got_ids, got_w = run(dg, x, None, k, score=score, renormalize=renorm, scale=2.0)
        assert np.array_equal(got_ids, ids)
        s = np.where(ids >= 0, around.route(x, None, k, score, renormalize=False)[1], 1.0)
        # each score to 5e-6 of itself and a unit of the subnormal range; with their sum in the quotient twice that
        far = 5e-6 + 2.0 * LEAST / s.min(axis=1, keepdims=True) if renorm else 5e-6 + LEAST / s
        assert np.all(np.abs(got_w - w) <= 2.0 * far * np.abs(w) + LEAST)


@pytest.mark.parametrize("E,k", PATHS)
def test_sigmoid_gradient_of_subnormal_scores(dg, E, k):
    print(f"case: sigmoid gradient of subnormal scores E={E} top_k={k}", flush=True)
    rng = np.random.default_rng(E * 5 + k)
    x = rng.uniform(-92.0, -88.0, (16, E)).astype(np.float32)
    ids, _, _ = around.route(x, None, k, "sigmoid")
    g = rng.standard_normal((16, k)).astype(np.float32)
    got = backward(dg, x, ids, g, score="sigmoid", renormalize=True, scale=1.0)
    ref = around.route_backward(x, ids, g, "sigmoid", True, 1.0)
    s = np.exp(np.take_along_axis(x, ids, axis=1).astype(np.float64))
    # a score is off by a unit of the subnormal range: its share of the sum twice that, then u's two terms
    far = 1e-5 + 8.0 * LEAST / s.min(axis=1, keepdims=True)
    assert np.all(np.abs(got - ref) <= far * np.abs(g).max(axis=1, keepdims=True))


@pytest.mark.parametrize("E,G", [(64, 1), (64, 4), (512, 8), (640, 1), (640, 20), (48, 8)])
def test_keys_of_infinity(dg, E, G):
    # +inf is above the largest finite key on either kernel; equal ones go to the lowest index
    print(f"case: route keys of +inf E={E} groups={G}", flush=True)
    x = np.tile(np.linspace(-1.0, 1.0, E, dtype=np.float32), (3, 1))
    bias = np.zeros(E, dtype=np.float32)
    bias[1], bias[3], bias[E - 1], bias[E - 4] = MOST, MOST, np.inf, np.inf
    kept = max(1, G // 2)
    for group_top in (1, 2):
        with np.errstate(invalid="ignore"):
            ids, w, _ = around.route(x, bias, 4, "sigmoid", G, kept, group_top)
        assert ids[0, 0] == E - 4 and ids[0, 1] == E - 1
        got_ids, got_w = run(dg, x, bias, 4, score="sigmoid", num_groups=G, topk_groups=kept, group_top=group_top)
        assert np.array_equal(got_ids, ids)
        assert np.all(np.abs(got_w - w) <= 5e-6 * w)


@pytest.mark.parametrize("E,G", [(64, 4), (512, 16), (640, 4), (96, 32), (30, 5)])
def test_group_scores_beyond_the_finite_range(dg, E, G):
    # the type's lowest value is no mask: two such keys sum to -2 MOST, which is below one of
    # them and still a score; two of MOST are above one of them
    print(f"case: group scores of +-2 MOST E={E} groups={G}", flush=True)
    per, kept, k = E // G, 2, 3
    x = np.tile(np.linspace(-1.0, 1.0, E, dtype=np.float32), (2, 1))
    cases = []
    low = np.full(E, -MOST, dtype=np.float32)
    cases.append(low)                                # nothing else: the lowest indices
    one = low.copy()                                 # the last group has one such key, the rest of it masked
    one[(G - 1) * per + 1:] = -np.inf
    cases.append(one)
    high = np.zeros(E, dtype=np.float32)             # group 2 holds MOST twice, groups 0 and 1 once
    high[0] = high[per] = high[2 * per] = high[2 * per + 1] = MOST
    cases.append(high)
    for at, bias in enumerate(cases):
        ids, w, _ = around.route(x, bias, k, "sigmoid", G, kept, 2)
        if at == 1:
            assert ids[0].tolist() == [0, 1, 2]      # groups G - 1 and 0; equal keys by index
            assert around.route(x, bias, 1, "sigmoid", G, 1, 2)[0][0, 0] == (G - 1) * per
        got_ids, _ = run(dg, x, bias, k, score="sigmoid", num_groups=G, topk_groups=kept, group_top=2)
        assert np.array_equal(got_ids, ids), at
        ids, _, _ = around.route(x, bias, 1, "sigmoid", G, 1, 2)
        got_ids, _ = run(dg, x, bias, 1, score="sigmoid", num_groups=G, topk_groups=1, group_top=2)
        assert np.array_equal(got_ids, ids), at


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(2, 1)] + PATHS)
def test_gradient_of_a_choice_that_takes_nearly_all(dg, E, k, score, renorm):
    # one expert's share is 1 - e^-5 to 1 - e^-38: its gradient is its share times what the others have
    print(f"case: gradient of a dominant choice {score} E={E} top_k={k} renormalize={renorm}", flush=True)
    rng = np.random.default_rng(E * 7 + k)
    T, scale = 34, 1.5
    x = rng.standard_normal((T, E)).astype(np.float32) - (40.0 if score == "sigmoid" else 0.0)
    x[np.arange(T), rng.integers(0, E, T)] += np.linspace(5.0, 38.0, T).astype(np.float32)
    x[5, 0] = x[5, 1] = x[5].max()                       # two of the highest
    x[7, x[7] < x[7].max()] = -np.inf                    # nothing beside it
    ids, _, _ = around.route(x, None, k, score)
    g = rng.standard_normal((T, k)).astype(np.float32)
    got = backward(dg, x, ids, g, score=score, renormalize=renorm, scale=scale)
    xd = x.astype(np.float64)
    p = 1.0 / (1.0 + np.exp(-xd)) if score == "sigmoid" else np.exp(xd - xd.max(axis=1, keepdims=True))
    if score == "softmax":
        p /= p.sum(axis=1, keepdims=True)
    want, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        i = ids[t][ids[t] >= 0]
        gt, pt = g[t, :i.size].astype(np.float64), p[t, i]
        if renorm:
            pt = pt / pt.sum()
        for j in range(i.size):
            rest = np.arange(i.size) != j
            if renorm:                                   # sums of what is not j, never 1 - share
                less = pt[rest].sum()
            elif score == "softmax":
                less = np.delete(p[t], i[j]).sum()
            else:
                less = 1.0
            others = pt[rest] if renorm or score == "softmax" else 0.0 * pt[rest]
            own = 1.0 / (1.0 + np.exp(xd[t, i[j]])) if score == "sigmoid" else 1.0
            want[t, i[j]] = scale * own * pt[j] * (gt[j] * less - (others * gt[rest]).sum())
            size[t, i[j]] = scale * own * pt[j] * (abs(gt[j]) * less + (others * np.abs(gt[rest])).sum())
        if score == "softmax" and not renorm:
            free = np.setdiff1d(np.arange(E), i)
            want[t, free] = -scale * p[t, free] * (pt * gt).sum()
            size[t, free] = scale * p[t, free] * (pt * np.abs(gt)).sum()
    # x - top rounds to 2^-24 of at most 45, 3e-6 in each of a product's two shares; the rest as above.
    # Subnormal scores stand a unit of 2^-149 apart
    assert np.all(np.abs(got - want) <= 2e-5 * size + 4.0 * LEAST)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", PATHS)
def test_a_nan_gradient_stays_one(dg, E, k, score, renorm):
    # whichever bits it has; and a token of masked experts only has none
    print(f"case: route gradient of NaN {score} E={E} top_k={k} renormalize={renorm}", flush=True)
    rng = np.random.default_rng(E)
    x = rng.standard_normal((6, E)).astype(np.float32)
    x[5] = -np.inf
    x[4, ::2] = -np.inf
    ids, _, _ = around.route(x, None, k, score)
    g = rng.standard_normal((6, k)).astype(np.float32)
    bits = g.view(np.uint32)
    bits[0, 1], bits[1, 0], bits[2, 2], bits[5] = 0x7FFFFFFF, 0x7FC00000, 0xFFFFFFFF, 0x7FFFFFFF
    got = backward(dg, x, ids, g, score=score, renormalize=renorm, scale=1.0)
    for t, j in ((0, 1), (1, 0), (2, 2)):
        assert np.isnan(got[t, ids[t, j]])
        if score == "softmax" and not renorm:
            assert np.isnan(got[t]).all()
    assert np.isfinite(got[3:]).all() and np.all(got[5] == 0.0) and np.all(got[4, ::2] == 0.0)
