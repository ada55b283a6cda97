"""The 4-bit products whose sums are exact in fp32 (tests/exact4.py), on the CPU: that
they agree with the oracle's weights, that their sums fit, and that a mistake in the
reference shows in the bf16 results."""
import numpy as np
import pytest
import torch

from oracle import layer
from tests.exact4 import FORMS, decode, generator, of_expert, product, quarters, weights, whole


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_the_weights_are_the_oracle_s(form):
    args = weights(generator(0, "cpu"), form, (3,), 5, 384)
    for e in range(3):
        a = of_expert(args, e)
        want = layer.fp4_weights(a[0].numpy(), a[1].numpy()) if form == "fp4" else \
            layer.int4_weights(a[0].numpy(), a[1].double().numpy(), None if a[2] is None else a[2].numpy())[0]
        assert np.array_equal(decode(form, *a).numpy(), want)


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_sums_fit_fp32_and_a_mistake_shows(form):
    """At the largest K: all magnitudes together are below 2^22 units, and leaving out 8 values of K, taking the scale of
    the block beside, or another 8 values' codes gives other bf16 values in nearly every row."""
    g = generator(1, "cpu")
    N, K, M = 64, 16512, 4
    args = weights(g, form, (), N, K)
    x, c, w = whole(g, M, K), quarters(g, M, N), decode(form, *args)
    unit = 0.25 if form == "fp4" else 0.5
    most = w.abs().max() if form == "fp4" else 60.0
    assert float(most) * 2 * K + 32 < 2 ** 24 * unit / 2
    assert torch.equal(w / unit, (w / unit).round())
    want = product(x, w, c)
    assert torch.equal(want.float(), (x.float() @ w.float().t() + c.float()).to(torch.bfloat16).float())
    for at in (0, 8192, K - 128, K - 8):
        less = w.clone()
        less[:, at:at + 8] = 0
        assert (product(x, less, c) != want).float().mean() > 0.3, at
        moved = w.clone()
        moved[:, at:at + 8] = w[:, (at + 128) % K:(at + 128) % K + 8]
        assert (product(x, moved, c) != want).float().mean() > 0.3, at
    scales = [args[1].clone(), *args[2:]]
    scales[0][-1] = scales[0][0]
    assert (product(x, decode(form, args[0], *scales), c) != want).float().mean() > 0.3
