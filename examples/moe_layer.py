"""A mixture-of-experts layer on this library's calls, served and trained.

    y = shared projection of x (FP8 dense product) with low-rank adapters per request
    ids, weights = router(y);  d = y + sum_j weights_j * expert_{ids_j}(x)

serve()       runs it for a batch of tokens, over the masked layout (decoding: nothing
              depends on the host, so the step can be captured in a HIP graph) or the
              contiguous one (prefill);
serve_few()   runs it for a few tokens on 4-bit weights and unquantised activations,
              the experts straight from the router's choices;
train()       adds the gradients of a given d: the expert weights' (K-grouped product),
              the router weights' and the router's logits';
train_step()  adds the router's balance loss to it, and clips all gradients together.

Run as a program it checks both against float64 and prints the differences:
python examples/moe_layer.py"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_grouped_gemm_nt_amd as dg  # noqa: E402


def quantise_blocks(w):
    """Weights [..., N, K] as e4m3 codes with one fp32 scale per 128 x 128 block (once, at load time)."""
    *lead, N, K = w.shape
    n = -(-N // 128)
    padded = torch.zeros(*lead, n * 128, K, device=w.device)
    padded[..., :N, :] = w.float()
    blocks = padded.view(*lead, n, 128, K // 128, 128)
    amax = blocks.abs().amax(dim=(-3, -1))
    sf = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = (blocks / sf[..., :, None, :, None]).clamp(-448.0, 448.0).view(*lead, n * 128, K)[..., :N, :]
    return q.to(torch.float8_e4m3fn).contiguous(), sf.contiguous()


FP4 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise_fp4(w):
    """Weights [..., N, K] as packed E2M1 codes with one power-of-two scale per 32 values of K (once, at load time):
    (b uint8 [..., N, K/2], sfb int32 [..., K/128, N], the weights that these stand for)."""
    *lead, N, K = w.shape
    blocks = w.float().view(*lead, N, K // 32, 32)
    amax = blocks.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
    e = torch.floor(torch.log2(amax)) - 2                        # the largest value lies in [4, 8)
    v = (blocks * torch.exp2(-e)).clamp(-6.0, 6.0)
    levels = FP4.to(w.device)
    code = torch.bucketize(v.abs(), (levels[1:] + levels[:-1]) / 2)
    stand_for = (levels[code] * torch.sign(v) * torch.exp2(e)).view(*lead, N, K)
    code = (code + 8 * (v < 0)).to(torch.uint8).view(*lead, N, K // 2, 2)
    sf = (e + 127).to(torch.uint8).view(*lead, N, K // 128, 4).transpose(-3, -2).contiguous()
    return (code[..., 0] | code[..., 1] << 4).contiguous(), sf.view(torch.int32).squeeze(-1).contiguous(), stand_for


class MoELayer:
    """The weights of one layer: shared [H][H], router [E][H], experts [E][H][H], adapters [L][R][H] and [L][H][R]."""

    def __init__(self, shared, router, experts, lora_a, lora_b, top_k, groups=1, kept=1):
        self.shared, self.shared_sf = quantise_blocks(shared)
        self.experts, self.experts_sf = quantise_blocks(experts)
        self.shared4, self.shared4_sf, _ = quantise_fp4(shared)
        self.experts4, self.experts4_sf, _ = quantise_fp4(experts)
        self.router = router.t().contiguous().float()
        self.lora_a, self.lora_b = lora_a.to(torch.bfloat16), lora_b.to(torch.bfloat16)
        self.top_k, self.groups, self.kept = top_k, groups, kept
        self.bias = torch.zeros(experts.shape[0], device=experts.device)

    def project(self, x, adapter_ids):
        """y = shared . x + adapters: the adapters' terms are the C of the dense call."""
        T, H = x.shape
        dev = x.device
        rows = torch.arange(T, dtype=torch.int32, device=dev)          # every token its own row
        a = torch.empty(T, H, dtype=torch.uint8, device=dev)
        sfa = torch.empty(H // 128, T, device=dev)
        dg.dg_m_grouped_scatter_fp8_contiguous(x, None, rows.view(T, 1), rows, a, sfa)
        y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        dg.dg_lora_bf16_nt(x, self.lora_a, self.lora_b, None, adapter_ids, None, y)
        dg.dg_fp8_gemm_nt(a, sfa, self.shared, self.shared_sf, y, y)
        return y

    def route(self, y):
        logits = y.float() @ self.router
        T = y.shape[0]
        ids = torch.empty(T, self.top_k, dtype=torch.int32, device=y.device)
        weights = torch.empty(T, self.top_k, device=y.device)
        dg.dg_route_topk(logits, self.bias, ids, weights, score="sigmoid", num_groups=self.groups,
                         topk_groups=self.kept, group_top=2)
        return logits, ids, weights

    def experts_contiguous(self, x, ids):
        """The experts' results for every choice: rows [M][H], and the maps."""
        T, H = x.shape
        dev, E = x.device, self.experts.shape[0]
        M = dg.dg_m_grouped_rows_bound(ids.numel(), E)
        i32 = dict(dtype=torch.int32, device=dev)
        layout, slot_of, counts = torch.empty(M, **i32), torch.empty(M, **i32), torch.empty(E, **i32)
        row_of = torch.empty_like(ids)
        dg.dg_m_grouped_layout_contiguous(ids, 0, layout, row_of, slot_of, counts)
        a = torch.empty(M, H, dtype=torch.uint8, device=dev)
        sfa = torch.empty(H // 128, M, device=dev)
        dg.dg_m_grouped_scatter_fp8_contiguous(x, None, row_of, slot_of, a, sfa)
        rows = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
        dg.dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, self.experts, self.experts_sf, None, rows, layout)
        return rows, row_of, slot_of, counts

    def experts_masked(self, x, ids, max_m):
        T, H = x.shape
        dev, E = x.device, self.experts.shape[0]
        i32 = dict(dtype=torch.int32, device=dev)
        masked_m, slot_of, row_of = torch.empty(E, **i32), torch.empty(E, max_m, **i32), torch.empty_like(ids)
        dg.dg_m_grouped_layout_masked(ids, 0, masked_m, row_of, slot_of)
        a = torch.empty(E, max_m, H, dtype=torch.uint8, device=dev)
        sfa = torch.empty(E, H // 128, max_m, device=dev)
        dg.dg_m_grouped_scatter_fp8_masked(x, None, row_of, slot_of, a, sfa)
        rows = torch.empty(E, max_m, H, dtype=torch.bfloat16, device=dev)
        dg.dg_m_grouped_fp8_gemm_nt_masked(a, sfa, self.experts, self.experts_sf, None, rows, masked_m,
                                           max(1, ids.numel() // E))
        return rows, row_of

    def serve(self, x, adapter_ids, max_m=None):
        """d [T][H]; with max_m over the masked layout (rows beyond max_m of an expert are dropped)."""
        y = self.project(x, adapter_ids)
        _, ids, weights = self.route(y)
        rows, row_of = self.experts_masked(x, ids, max_m) if max_m else self.experts_contiguous(x, ids)[:2]
        d = torch.empty_like(y)
        dg.dg_m_grouped_gather(rows, row_of, weights, y, d)
        return d

    def serve_few(self, x, adapter_ids):
        """d [T][H] of a few tokens, on the 4-bit weights: six launches, no rows moved or quantised."""
        T, H = x.shape
        k = self.top_k
        y = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
        dg.dg_lora_bf16_nt(x, self.lora_a, self.lora_b, None, adapter_ids, None, y)
        dg.dg_bf16_fp4_gemv_nt(x, self.shared4, self.shared4_sf, y, y)
        _, ids, weights = self.route(y)
        rows = torch.empty(T * k, H, dtype=torch.bfloat16, device=x.device)
        dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x, ids, 0, self.experts4, self.experts4_sf, None, rows)
        row_of = torch.arange(T * k, dtype=torch.int32, device=x.device).view(T, k)
        d = torch.empty_like(y)
        dg.dg_m_grouped_gather(rows, row_of, weights, y, d)
        return d

    def train_step(self, x, adapter_ids, grad_d, seq_starts=None, balance=0.01, max_norm=1.0):
        """(d, {"experts", "logits"}: the clipped gradients with the balance loss's, their norm before, the loss per
        sequence, the experts' counts)."""
        d, grad_experts, grad_logits, (logits, ids, _, _) = self.train(x, adapter_ids, grad_d)
        S = 1 if seq_starts is None else seq_starts.numel() - 1
        loss = torch.empty(S, device=x.device)
        counts = torch.empty(S, logits.shape[1], dtype=torch.int32, device=x.device)
        dg.dg_route_balance(logits, ids, seq_starts, loss, counts, score="sigmoid", scale=balance)
        dg.dg_route_balance_backward(logits, counts, seq_starts, None, grad_logits, grad_logits, self.top_k,
                                     score="sigmoid", scale=balance)
        norm = torch.empty(1, device=x.device)
        grads = [grad_experts, grad_logits]
        dg.dg_grad_norm(grads, norm)
        dg.dg_grad_clip(grads, grads, norm, max_norm)
        return d, {"experts": grad_experts, "logits": grad_logits}, norm, loss, counts

    def train(self, x, adapter_ids, grad_d):
        """(d, gradients of experts [E][H][H] fp32, of the router's logits [T][E], choices) for grad_d bf16 [T][H]."""
        T, H = x.shape
        dev, E, k = x.device, self.experts.shape[0], self.top_k
        y = self.project(x, adapter_ids)
        logits, ids, weights = self.route(y)
        rows, row_of, slot_of, counts = self.experts_contiguous(x, ids)
        d = torch.empty_like(y)
        dg.dg_m_grouped_gather(rows, row_of, weights, y, d)
        grad_weights = torch.empty(T, k, device=dev)
        dg.dg_m_grouped_gather_weight_grad(rows, row_of, grad_d, grad_weights)
        grad_logits = torch.empty_like(logits)
        dg.dg_route_topk_backward(logits, ids, grad_weights, grad_logits, score="sigmoid")
        # experts: sum over an expert's rows of (weight * grad_d) x^T, K-grouped over the segments in use
        ks = [-(-n // 128) * 128 for n in counts.tolist()]
        K = sum(ks)
        ga = torch.empty(K, H, dtype=torch.uint8, device=dev)
        xa = torch.empty(K, H, dtype=torch.uint8, device=dev)
        gsf, xsf = torch.empty(K // 128, H, device=dev), torch.empty(K // 128, H, device=dev)
        dg.dg_k_grouped_scatter_fp8(grad_d, weights, slot_of[:K], k, ga, gsf)
        dg.dg_k_grouped_scatter_fp8(x, None, slot_of[:K], k, xa, xsf)
        grad_experts = torch.empty(E, H, H, device=dev)
        dg.dg_k_grouped_fp8_gemm_tn_contiguous(ga, gsf, xa, xsf, None, grad_experts, ks)
        return d, grad_experts, grad_logits, (logits, ids, weights, grad_weights)


def make(H=512, E=16, L=5, R=16, top_k=4, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*s, scale=1.0):
        return torch.randn(*s, device="cuda", generator=g) * scale

    w = dict(shared=randn(H, H, scale=H ** -0.5), router=randn(E, H, scale=H ** -0.5),
             experts=randn(E, H, H, scale=H ** -0.5), lora_a=randn(L, R, H, scale=H ** -0.5),
             lora_b=randn(L, H, R, scale=R ** -0.5))
    return MoELayer(top_k=top_k, groups=4, kept=2, **w), w, g


def tokens(g, T, H, L):
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    return x, torch.randint(-1, L, (T,), device="cuda", generator=g, dtype=torch.int32)


def reference(w, x, adapter_ids, ids, weights):
    """d in float64 for the layer's own choice of experts, from the unquantised weights."""
    x = x.double()
    y = x @ w["shared"].double().t()
    for i in range(w["lora_a"].shape[0]):
        t = adapter_ids == i
        y[t] += x[t] @ w["lora_a"][i].to(torch.bfloat16).double().t() @ w["lora_b"][i].to(torch.bfloat16).double().t()
    d = y.clone()
    for e in range(w["experts"].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        d[t] += weights[t, j].double().unsqueeze(1) * (x[t] @ w["experts"][e].double().t())
    return d


def relative(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def check(T=300, seed=0):
    """{what: relative difference from float64}; e4m3 operands account for about 0.04."""
    layer, w, g = make(seed=seed)
    H, E = w["shared"].shape[0], w["experts"].shape[0]
    x, adapter_ids = tokens(g, T, H, w["lora_a"].shape[0])
    grad_d = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    d, grad_experts, grad_logits, (logits, ids, weights, grad_weights) = layer.train(x, adapter_ids, grad_d)
    out = {"d": relative(d, reference(w, x, adapter_ids, ids, weights)),
           "served, contiguous": relative(layer.serve(x, adapter_ids), d),
           "served, masked": relative(layer.serve(x, adapter_ids, max_m=T), d)}
    want = torch.zeros(E, H, H, dtype=torch.double, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        want[e] = (weights[t, j].double().unsqueeze(1) * grad_d[t].double()).t() @ x[t].double()
    out["gradient of the experts"] = relative(grad_experts, want)
    # from the layer's own gradient of the weights: a token's logits get differences
    # of these, in which the e4m3 error of each stands out
    free = logits.double().requires_grad_(True)
    s = torch.sigmoid(free).gather(1, ids.long())
    ((s / s.sum(1, keepdim=True)) * grad_weights.double()).sum().backward()
    out["gradient of the logits"] = relative(grad_logits, free.grad)
    # the 4-bit weights, from what they stand for
    few = dict(w, shared=quantise_fp4(w["shared"])[2], experts=quantise_fp4(w["experts"])[2])
    t = min(T, 32)
    y = x[:t].double() @ few["shared"].double().t()
    for i in range(few["lora_a"].shape[0]):
        on = adapter_ids[:t] == i
        y[on] += x[:t][on].double() @ few["lora_a"][i].to(torch.bfloat16).double().t() @ \
            few["lora_b"][i].to(torch.bfloat16).double().t()
    _, ids4, weights4 = layer.route(y.to(torch.bfloat16))
    out["served, 4-bit"] = relative(layer.serve_few(x[:t], adapter_ids[:t]),
                                    reference(few, x[:t], adapter_ids[:t], ids4, weights4))
    # the balance loss of sequences of a third and two thirds, by differentiation
    starts = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    _, grads, norm, loss, counts = layer.train_step(x, adapter_ids, grad_d, starts, balance=0.1, max_norm=1e9)
    free = logits.double().requires_grad_(True)
    p = torch.sigmoid(free)
    p = p / p.sum(1, keepdim=True)
    wanted = []
    for a, b in ((0, T // 3), (T // 3, T)):
        f = torch.bincount(ids[a:b].flatten(), minlength=E).double() * E / (layer.top_k * max(1, b - a))
        wanted.append(0.1 * (f * p[a:b].sum(0)).sum() / max(1, b - a))
    sum(wanted).backward()
    out["balance loss"] = relative(loss, torch.stack(wanted).detach())
    out["gradient with the balance loss"] = relative(grads["logits"], grad_logits.double() + free.grad)
    out["norm"] = relative(norm, torch.sqrt(grads["experts"].double().square().sum() +
                                            grads["logits"].double().square().sum()).view(1))
    return out


if __name__ == "__main__":
    for what, far in check().items():
        print(f"{what}: {far:.4f}")
