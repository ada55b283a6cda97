"""The fp64 oracle of the balance loss, the 4-bit weights and the gradients'
clipping: values worked out by hand, and its gradient against differences.  No GPU."""
import numpy as np
import pytest

from oracle import layer


def test_balance_by_hand():
    x = np.log(np.array([[1.0, 1.0, 2.0], [1.0, 3.0, 0.0 + 1e-300]]))
    ids = np.array([[2, 0], [1, -1]])
    loss, counts = layer.balance(x, ids, None, "softmax", scale=2.0)
    assert counts.tolist() == [[1, 1, 1]]
    # E / (k n^2) = 3 / 8; sums of shares (1/4 + 1/4, 1/4 + 3/4, 1/2) with counts of 1: 2
    assert np.allclose(loss, [2.0 * 3 / 8 * 2.0])
    loss, counts = layer.balance(x, ids, [0, 1, 1, 2], "softmax")
    assert counts.tolist() == [[1, 0, 1], [0, 0, 0], [0, 1, 0]]
    assert np.allclose(loss, [3 / 2 * 0.75, 0.0, 3 / 2 * 0.75])


def test_equal_shares_give_the_scale():
    T, E, k = 12, 6, 2
    ids = np.stack([np.arange(T) % E, (np.arange(T) + 3) % E], axis=1)
    for score in ("softmax", "sigmoid"):
        loss, counts = layer.balance(np.zeros((T, E)), ids, None, score, scale=0.3)
        assert np.allclose(loss, 0.3) and (counts == T * k // E).all()


def test_masks():
    x = np.array([[-np.inf, np.nan, 0.0], [-np.inf] * 3, [np.inf, 0.0, 1.0], [-700.0, -701.0, -np.inf]])
    for score in ("softmax", "sigmoid"):
        p, _ = layer.shares(x, score)
        assert p[0].tolist() == [0.0, 0.0, 1.0] and p[1].tolist() == [0.0] * 3
        assert np.isclose(p[3, 0], 1 / (1 + np.exp(-1.0))) and p[3, 2] == 0.0
    assert layer.shares(x, "softmax")[0][2].tolist() == [1.0, 0.0, 0.0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_by_differences(score):
    rng = np.random.default_rng(0)
    T, E, k = 7, 5, 2
    x = rng.standard_normal((T, E))
    x[2, 1] = -np.inf
    ids = np.argsort(-x, axis=1)[:, :k]
    starts, grad_loss = [1, 4, 4, 6], np.array([1.5, 2.0, -0.5])
    _, counts = layer.balance(x, ids, starts, score, 0.7)
    c = rng.standard_normal((T, E))
    got, _ = layer.balance_backward(x, counts, starts, grad_loss, c, k, score, 0.7)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if x[t, e] == -np.inf:
                assert got[t, e] == c[t, e]
                continue
            v = []
            for d in (h, -h):
                y = x.copy()
                y[t, e] += d
                v.append(float(layer.balance(y, ids, starts, score, 0.7)[0] @ grad_loss))
            assert abs((v[0] - v[1]) / (2 * h) + c[t, e] - got[t, e]) < 1e-8, (t, e)


def test_weights_by_hand():
    b = np.zeros((1, 64), dtype=np.uint8)
    b[0, 0], b[0, 16], b[0, 63] = 0x71, 0xF2, 0x40               # k = 0, 1; 32, 33; 126, 127
    sfb = np.array([[127 | 128 << 8 | 126 << 16 | 120 << 24]], dtype=np.int32)
    w = layer.fp4_weights(b, sfb)
    assert w[0, 0] == 0.5 and w[0, 1] == 6.0 and w[0, 32] == 2.0 and w[0, 33] == -12.0
    assert w[0, 126] == 0.0 and w[0, 127] == 2.0 * 2.0 ** -7 and np.count_nonzero(w) == 5
    w, most = layer.int4_weights(b, np.array([[0.5], [2.0], [1.0], [1.0]]), np.array([[1], [2], [0], [4]], dtype=np.uint8))
    assert w[0, 0] == 0.0 and w[0, 1] == 3.0 and w[0, 2] == -0.5
    assert w[0, 32] == 0.0 and w[0, 33] == 26.0 and w[0, 127] == 0.0 and w[0, 126] == -4.0
    assert most[0, 33] == 34.0
    assert layer.int4_weights(b, np.ones((1, 1)), None)[0][0, :2].tolist() == [-7.0, -1.0]


def test_norm_and_factor():
    assert layer.grad_norm([np.array([3.0]), np.array([[0.0, -4.0]]), np.zeros(0)]) == 5.0
    assert layer.grad_factor(5.0, 10.0) == 1.0 and np.isclose(layer.grad_factor(5.0, 1.0), 1 / 5.000001)
