"""The fp64 oracle of the operators around the products: values worked out by
hand, and its gradient against differences.  No GPU."""
import numpy as np
import pytest

import oracle
from oracle import around


def test_route_by_hand():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w, margin = around.route(x, None, 2, "softmax", renormalize=False)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]]) and np.isclose(margin[0], 0.125)
    ids, w, _ = around.route(x, None, 2, "softmax", renormalize=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]])
    bias = np.array([1.0, 0.0, 0.0, 1.0])           # the bias moves the choice and not the weights
    ids, w, margin = around.route(x, bias, 2, "softmax", renormalize=False)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, 0.125) and margin[0] == 0.0
    ids, _, _ = around.route(x, None, 1, "sigmoid", num_groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[2]]
    y = np.array([[3.0, -9.0, 2.0, 2.0]])           # groups by their highest, or by the sum of two
    assert around.route(y, None, 1, "sigmoid", 2, 1, 1)[0].tolist() == [[0]]
    assert around.route(y, None, 1, "sigmoid", 2, 1, 2)[0].tolist() == [[2]]


def test_route_masks():
    x = np.array([[-np.inf, np.nan, 0.0], [-np.inf] * 3])
    for score in ("softmax", "sigmoid"):
        ids, w, _ = around.route(x, None, 2, score)
        assert ids.tolist() == [[2, -1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]
        assert np.all(around.route_backward(x, ids, np.ones((2, 2)), score, True, 1.0) == 0.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_by_differences(score, renorm):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 9))
    ids, _, _ = around.route(x, None, 3, score)
    ids[1, 2] = -1
    g = rng.standard_normal((4, 3))
    got = around.route_backward(x, ids, g, score, renorm, 1.7)
    h = 1e-5
    for e in range(9):
        d = np.zeros_like(x)
        d[:, e] = h
        ref = ((around.route_weights(x + d, ids, score, renorm, 1.7) -
                around.route_weights(x - d, ids, score, renorm, 1.7)) / (2 * h) * g).sum(axis=1)
        assert np.allclose(got[:, e], ref, atol=1e-8)


def test_layouts_by_hand():
    ids = np.array([[3, 4], [4, 9], [4, 3]])
    layout, row, slot, counts = around.layout_contiguous(ids, 3, 2, 384)
    assert counts.tolist() == [2, 3] and row.tolist() == [[0, 128], [129, -1], [130, 1]]
    assert slot[[0, 1, 2, 128, 129, 130, 131]].tolist() == [0, 5, -1, 1, 2, 4, -1]
    assert layout[[0, 1, 2, 128, 130, 131, 383]].tolist() == [0, 0, -1, 1, 1, -1, -1]
    oracle_layout = layout.copy()
    assert set(oracle_layout.tolist()) == {-1, 0, 1}
    mm, row, slot = around.layout_masked(ids, 3, 2, 2)
    assert mm.tolist() == [2, 2] and row.tolist() == [[0, 2], [3, -1], [-1, 1]] and slot.tolist() == [[0, 5], [1, 2]]


def test_layout_fits_the_products_contract():
    import moe_grouped_gemm_nt_amd as dg
    rng = np.random.default_rng(3)
    ids = rng.integers(0, 12, (500, 4))
    layout, _, _, _ = around.layout_contiguous(ids, 2, 8, around.rows_bound(2000, 8))
    dg.dg_check_grouped_layout(layout, 8)


def test_block_scales_and_steps():
    amax = np.array([0.0, 448.0, 449.0, 1.0, 2.0 ** -120])
    assert around.block_scales(amax, False).tolist() == [1.0, 1.0, 449.0 / 448.0, 1.0 / 448.0, 2.0 ** -100 / 448.0]
    assert around.block_scales(amax, True).tolist() == [1.0, 1.0, 2.0, 2.0 ** -8, 2.0 ** -108]
    v = np.unique(np.abs(oracle.E4M3_VALUES[np.isfinite(oracle.E4M3_VALUES)]))
    assert np.array_equal(np.diff(v), around.e4m3_step(v[:-1]))


def test_gather_and_adapters_by_hand():
    rows = np.array([[1.0, 2.0], [10.0, 20.0], [100.0, 200.0]], dtype=np.float32)
    at = np.array([[0, 2], [-1, 3]])
    w = np.array([[2.0, 0.5], [9.0, 9.0]])
    out, mag = around.gather(rows, at, w, np.array([[1.0, 1.0], [5.0, 6.0]]))
    assert out.tolist() == [[53.0, 105.0], [5.0, 6.0]] and mag.tolist() == out.tolist()
    g, _ = around.gather_weight_grad(rows, at, np.array([[1.0, -1.0], [1.0, 1.0]]))
    assert g.tolist() == [[-1.0, -100.0], [0.0, 0.0]]
    a, b = np.array([[[1.0, 2.0]]]), np.array([[[3.0], [4.0]]])
    out, _ = around.lora(np.array([[1.0, 1.0], [1.0, 0.0]]), a, b, [2.0], [0, -1], np.ones((2, 2)))
    assert out.tolist() == [[19.0, 25.0], [1.0, 1.0]]
