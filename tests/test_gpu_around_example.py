"""The example layer's gradients of the router, step by step against float64
with bounds of fp32 rounding only: each from the layer's own rows and weights."""
import numpy as np
import pytest
import torch

import examples.moe_layer as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 7, 300, 1000])
def test_router_gradients_of_the_example(T):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"case: the example's router gradients, {T} tokens", flush=True)
    layer, w, g = moe.make(seed=T + 1)
    H = w["shared"].shape[0]
    x, adapter_ids = moe.tokens(g, T, H, w["lora_a"].shape[0])
    grad_d = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    _, _, grad_logits, (logits, ids, weights, grad_weights) = layer.train(x, adapter_ids, grad_d)
    rows, row_of, _, _ = layer.experts_contiguous(x, ids)
    torch.cuda.synchronize()
    # weights' gradient: products of bf16 are exact in fp32, H additions in any order
    at = row_of.long()
    assert bool((at >= 0).all())
    terms = rows.double()[at] * grad_d.double().unsqueeze(1)
    ref = terms.sum(2)
    assert bool(((grad_weights.double() - ref).abs() <= H * 2.0 ** -24 * terms.abs().sum(2)).all())
    # logits': scores within 5e-7, sums of four of them, a few products; u = share (g - sum share g)
    free = logits.double().requires_grad_(True)
    s = torch.sigmoid(free).gather(1, ids.long())
    ((s / s.sum(1, keepdim=True)) * grad_weights.double()).sum().backward()
    most = grad_weights.double().abs().amax(1, keepdim=True)
    assert bool(((grad_logits.double() - free.grad).abs() <= 1e-5 * most).all())
    assert moe.relative(grad_logits, free.grad) < 1e-5
    want = s / s.sum(1, keepdim=True)
    assert float((weights.double() - want).abs().max()) < 5e-6
    assert np.isfinite(float(most.max()))
