"""The router over more tokens than one grid has threads for (2^32, sixteen or 64 to
a token): the last ones of 2^28 and 2^26 tokens, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import around

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    yield m
    torch.cuda.empty_cache()


# T, E, top_k, groups: sixteen lanes per token, then one wave (groups of two, or more than 16 choices)
CASES = [(2 ** 28 + 17, 2, 1, 1), (2 ** 26 + 9, 4, 1, 2), (2 ** 26 + 5, 18, 17, 1)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_more_tokens_than_a_grid(dg, case):
    T, E, k, G = case
    print(f"case: router over {T} tokens of {E} experts", flush=True)
    rng = np.random.default_rng(E)
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    far = [0, 1, T // 2, T - 20000, T - 2, T - 1]
    v = torch.from_numpy(rng.standard_normal((len(far), E)).astype(np.float32)).to(torch.bfloat16)
    logits[torch.tensor(far, device="cuda")] = v.cuda()
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -1.0, device="cuda")
    dg.dg_route_topk(logits, None, ids, w, score="sigmoid", num_groups=G, renormalize=False)
    torch.cuda.synchronize()
    ref_ids, ref_w, _ = around.route(v.float().numpy(), None, k, "sigmoid", num_groups=G, renormalize=False)
    assert np.array_equal(ids[far].cpu().numpy(), ref_ids)
    assert np.all(np.abs(w[far].cpu().numpy() - ref_w) <= 5e-6 * ref_w)
    assert int((ids[:, 0] < 0).sum()) == 0 and int((w <= 0.0).sum()) == 0
    grad = torch.full_like(logits, float("nan"))
    dg.dg_route_topk_backward(logits, ids, w, grad, score="sigmoid", renormalize=False)
    torch.cuda.synchronize()
    ref = around.route_backward(v.float().numpy(), ref_ids, w[far].cpu().numpy(), "sigmoid", False, 1.0)
    assert np.all(np.abs(grad[far].float().cpu().numpy() - ref) <= 1e-5 + 2.0 ** -8 * np.abs(ref))
    assert not bool(torch.isnan(grad).any())
