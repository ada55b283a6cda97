"""The operators around the expert products and the shared projection, as measured.

Four operators, each with its plain form in elementary torch operations and the
calls a user makes of this package:

  route      tokens' scores to experts: sigmoid or softmax scores, a balance bias,
             expert groups, top-k, weights (and the gradient of the logits)
  rows_out   tokens' rows to the experts' rows: the layout of the M-grouped products,
             each row quantised to e4m3 with 1x128 scales (masked and contiguous), or
             with 128x1 scales for the K-grouped weight-gradient product
  rows_back  the experts' bf16 rows back to the tokens: a weighted sum onto a residual
             (and the gradient of its weights)
  lora       low-rank adapters, one per token, added to a shared projection's result

``own`` false: plain torch, computed in 32 bits and rounded once at the end.
``own`` true: the package's kernels."""
import math

import torch

own = False

BLOCK = 128           # K values per scale, and rows per expert block of the contiguous layout
E4M3_MAX = 448.0
TINY = 2.0 ** -100    # the least block maximum a scale is made from


def _dg():
    import moe_grouped_gemm_nt_amd as dg
    return dg


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _route(T, E, top_k, score, num_groups=1, topk_groups=1, group_top=1, bias=False, dtype="float32",
           renormalize=True, scale=1.0, direction="forward", masked=0.0):
    return dict(op="route", T=T, E=E, top_k=top_k, score=score, num_groups=num_groups, topk_groups=topk_groups,
                group_top=group_top, bias=bias, dtype=dtype, renormalize=renormalize, scale=scale,
                direction=direction, masked=masked)


def _rows_out(form, T, top_k, experts, first, groups, K, max_m=0, weighted=False, pow2=False):
    return dict(op="rows_out", form=form, T=T, top_k=top_k, experts=experts, first=first, groups=groups, K=K,
                max_m=max_m, weighted=weighted, pow2=pow2)


def _rows_back(direction, T, top_k, experts, N, weighted=True, residual=False):
    return dict(op="rows_back", direction=direction, T=T, top_k=top_k, experts=experts, N=N, weighted=weighted,
                residual=residual)


def _lora(T, adapters, R, N, K, residual=True, runs=1, idle=0.0):
    return dict(op="lora", T=T, adapters=adapters, R=R, N=N, K=K, residual=residual, runs=runs, idle=idle)


def listed():
    return [
        # one decoding step of 64 requests: 256 experts in 8 groups of which 4 stay, 8 chosen; a few microseconds, all latency
        dict(_route(64, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5), name="route_decode"),
        # the same router over a prefill batch
        dict(_route(16384, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5), name="route_prefill"),
        # the gradient of a softmax router over a training batch of odd length, an expert count that is no power of
        # two, bf16 logits, some experts masked
        dict(_route(20479, 60, 4, "softmax", dtype="bfloat16", direction="backward", masked=0.02),
             name="route_backward_softmax"),
        # decoding, experts shared over 4 GPUs: this one's 32 experts of 128 take what comes to them (masked layout)
        dict(_rows_out("masked", 128, 8, 128, 32, 32, 7168, max_m=256), name="rows_out_masked_decode"),
        # the contiguous product's 8 experts and 8192 rows, fed from 4096 tokens with 2 experts each
        dict(_rows_out("contiguous", 4096, 2, 8, 0, 8, 7168, pow2=True), name="rows_out_contiguous"),
        # a prefill batch to 256 experts, 8 per token: 65536 rows
        dict(_rows_out("contiguous", 8192, 8, 256, 0, 256, 7168), name="rows_out_contiguous_large"),
        # training: the rows of the weight-gradient product of those 8 experts, weighted, scaled down the tokens
        dict(_rows_out("kgrouped", 4096, 2, 8, 0, 8, 4096, weighted=True), name="rows_out_kgrouped"),
        # the decoding step's way back: 8 expert rows to one per token, onto the shared expert's result
        dict(_rows_back("forward", 64, 8, 32, 7168, residual=True), name="rows_back_decode"),
        # the prefill batch's way back
        dict(_rows_back("forward", 8192, 8, 256, 7168), name="rows_back_large"),
        # training: the gradient of the weights, an odd number of tokens and of columns
        dict(_rows_back("weight_grad", 4095, 2, 8, 7165), name="rows_back_weight_grad"),
        # decoding with many adapters beside the decode projection's 2112 x 7168: nearly every request its own adapter
        dict(_lora(64, 48, 16, 2112, 7168, idle=0.1), name="lora_decode"),
        # prefill: a few long requests, each with its adapter, beside a 4096 x 7168 projection
        dict(_lora(8192, 8, 64, 4096, 7168, runs=500), name="lora_prefill"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, mostly odd."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n if n < 4 or rng.random() < 0.25 and n % 1024 else n | 1))


_KS = [128, 256, 384, 640, 896, 1024, 1408, 2048, 4096, 4224, 7168, 8192, 16384]
_NS = [1, 24, 100, 129, 513, 1000, 2047, 2112, 4096, 7165, 7168, 7424, 16384]


def _drawn(rng):
    op = rng.choice(["route", "route", "rows_out", "rows_out", "rows_out", "rows_back", "rows_back", "lora", "lora"])
    if op == "route":
        E = rng.choice([8, 16, 48, 60, 64, 96, 128, 160, 256, 320, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 3, 4, 8, 16) if E % g == 0 and E // g >= 2])
        kept = rng.randint((groups + 1) // 2, groups)
        top_k = min(rng.choice([1, 2, 3, 4, 6, 8, 8, 10]), kept * (E // groups))
        score = rng.choice(["sigmoid", "softmax"])
        return _route(_log_int(rng, 1, 32768), E, top_k, score, groups, kept, rng.choice([1, 2]),
                      bias=rng.random() < 0.5, dtype=rng.choice(["float32", "bfloat16"]),
                      renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                      direction=rng.choice(["forward", "forward", "backward"]), masked=rng.choice([0.0, 0.0, 0.05]))
    if op == "rows_out":
        form = rng.choice(["contiguous", "contiguous", "masked", "kgrouped"])
        groups = rng.choice([1, 3, 8, 16, 31, 32, 64, 160, 256])
        share = rng.choice([1, 1, 2, 4])
        top_k = min(rng.choice([1, 2, 4, 6, 8]), groups * share)
        T = _log_int(rng, 1, 512 if form == "masked" else 8192)
        K = rng.choice(_KS)
        max_m = 0
        if form == "masked":   # about twice the mean, so that the fullest experts may run over
            max_m = max(4, _log_int(rng, 1, 2) * T * top_k // (groups * share))
            max_m = min(max_m + rng.randint(0, 64), T + 1)
        return _rows_out(form, T, top_k, groups * share, groups * rng.randrange(share), groups, K, max_m,
                         weighted=rng.random() < 0.4, pow2=rng.random() < 0.4)
    if op == "rows_back":
        return _rows_back(rng.choice(["forward", "forward", "weight_grad"]), _log_int(rng, 1, 8192),
                          rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([8, 16, 31, 64, 256]), rng.choice(_NS),
                          weighted=rng.random() < 0.7, residual=rng.random() < 0.5)
    T = _log_int(rng, 1, 8192)
    adapters = rng.choice([1, 2, 5, 8, 20, 32, 64])
    return _lora(T, adapters, rng.choice([8, 16, 24, 32, 64, 128]), rng.choice(_NS), rng.choice(_KS),
                 residual=rng.random() < 0.7, runs=rng.choice([1, 1, 40, 500]), idle=rng.choice([0.0, 0.1, 0.5]))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), work(c)["bytes"])
    while True:
        c = _drawn(rng)
        if work(c)["bytes"] <= most[c["op"]]:
            return c


def _bound_rows(c):
    """Rows that the contiguous layout of c can need, however the tokens choose."""
    n = c["T"] * c["top_k"]
    return (n + (BLOCK - 1) * min(c.get("groups", c["experts"]), n)) // BLOCK * BLOCK


def work(c):
    T = c["T"]
    if c["op"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        back = c["direction"] == "backward"
        n = T * c["E"] * size * (2 if back else 1) + T * c["top_k"] * 8 + (c["E"] * 4 if c["bias"] and not back else 0)
        return {"bytes": n, "flops": 8 * T * c["E"]}
    if c["op"] == "rows_out":
        n = T * c["top_k"]
        live = n * c["groups"] / c["experts"]                    # rows that come to this GPU's experts
        tokens = T * (1 - (1 - c["groups"] / c["experts"]) ** c["top_k"])
        K = c["K"]
        moved = tokens * K * 2 + live * K * (1 + 4 / BLOCK) + (n * 4 if c["weighted"] else 0)
        if c["form"] == "kgrouped":
            return {"bytes": tokens * K * 2 + _bound_rows(c) * (K * (1 + 4 / BLOCK) + 4) + (n * 4 if c["weighted"] else 0),
                    "flops": 3 * live * K}
        rows = _bound_rows(c) * 2 if c["form"] == "contiguous" else c["groups"] * (c["max_m"] + 1)
        return {"bytes": moved + n * 8 + rows * 4, "flops": 3 * live * K}
    if c["op"] == "rows_back":
        n, N = T * c["top_k"], c["N"]
        rows = n * 0.95                                          # a few slots have no row here
        if c["direction"] == "weight_grad":
            return {"bytes": rows * N * 2 + T * N * 2 + n * 8, "flops": 2 * rows * N}
        return {"bytes": rows * N * 2 + T * N * 2 * (2 if c["residual"] else 1) + n * (8 if c["weighted"] else 4),
                "flops": 2 * rows * N}
    K, N, R, L = c["K"], c["N"], c["R"], c["adapters"]
    runs = max(1.0, T / c["runs"])
    used = L * (1 - (1 - 1 / L) ** runs)                         # adapters that some token has
    live = T * (1 - c["idle"])
    n = live * K * 2 + T * N * 2 * (2 if c["residual"] else 1) + used * R * (K + N) * 2 + T * 4 + L * 4
    return {"bytes": n, "flops": 2 * live * R * (K + N)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _undecided(logits, bias, c):
    """Tokens whose choice hangs on the rounding of 32-bit scores: two different experts' (or groups') scores
    within a few units in the last place of one another, at a place where their order shows."""
    x = logits.double()
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1).nan_to_num()
    key = s if bias is None else s + bias.double()
    key = key.masked_fill(torch.isinf(x), -math.inf)
    T, E, G = c["T"], c["E"], c["num_groups"]
    same = x if bias is None else x + 7.0 * bias.double()       # equal only where the scores are equal for certain

    def close(v, tag, n):
        order = v.sort(dim=1, descending=True, stable=True)
        a, b = order.values[:, :n], order.values[:, 1:n + 1]
        ta, tb = tag.gather(1, order.indices[:, :n]), tag.gather(1, order.indices[:, 1:n + 1])
        a = a[:, :b.shape[1]]
        near = ((a - b) <= 4e-6 * (a.abs() + b.abs())) & torch.isfinite(a) & torch.isfinite(b)
        return (near & (ta[:, :b.shape[1]] != tb)).any(1)

    bad = torch.zeros(T, dtype=torch.bool, device=x.device)
    if G > 1:
        per = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        gs = per.masked_fill(per == -math.inf, 0.0).sum(2).masked_fill(per[:, :, 0] == -math.inf, -math.inf)
        if c["topk_groups"] < G:
            bad |= close(gs, gs + torch.arange(G, device=x.device), c["topk_groups"])
        kept = gs.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = key.masked_fill(~mask.repeat_interleave(E // G, 1), -math.inf)
    if c["top_k"] < E:
        bad |= close(key, same, c["top_k"])
    else:
        bad |= close(key, same, E - 1)
    return bad


def _choices(g, T, experts, top_k, dev):
    """Expert ids [T][top_k] without repeats, some experts liked more than others."""
    liking = torch.randn(experts, device=dev, generator=g) * 0.5
    noise = torch.rand(T, experts, device=dev, generator=g).clamp_(1e-7, 1 - 1e-7)
    return (liking - torch.log(-torch.log(noise))).topk(top_k, 1).indices.to(torch.int32)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T = c["T"]
    s = {"c": c}
    if c["op"] == "route":
        E = c["E"]
        dtype = getattr(torch, c["dtype"])
        bias = torch.randn(E, device=dev, generator=g) * 0.05 if c["bias"] else None

        def fresh(n):
            x = torch.randn(n, E, device=dev, generator=g) * 1.5
            if c["masked"]:
                x.masked_fill_(torch.rand(n, E, device=dev, generator=g) < c["masked"], -math.inf)
            return x.to(dtype)

        x = fresh(T)
        if c["masked"]:
            x[T // 2] = -math.inf                                # a token that no expert may take
        for _ in range(12):
            bad = _undecided(x, bias, c).nonzero().view(-1)
            if not bad.numel():
                break
            x[bad] = fresh(bad.numel())
        s.update(logits=x.contiguous(), bias=bias)
        s["ids"] = torch.empty(T, c["top_k"], dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(T, c["top_k"], dtype=torch.float32, device=dev)
        if c["direction"] == "backward":
            ids, _ = _route_plain(s)
            s["ids"] = ids
            s["grad_weights"] = torch.randn(T, c["top_k"], device=dev, generator=g)
            s["grad_logits"] = torch.empty_like(s["logits"])
        return s
    if c["op"] in ("rows_out", "rows_back"):
        experts, k = c["experts"], c["top_k"]
        s["ids"] = _choices(g, T, experts, k, dev)
        w = torch.rand(T, k, device=dev, generator=g) + 0.05
        s["weights"] = (w / w.sum(1, keepdim=True)) if c["weighted"] else None
    if c["op"] == "rows_out":
        K, G = c["K"], c["groups"]
        x = torch.randn(T, K, device=dev, generator=g)
        x *= torch.exp(0.5 * torch.randn(1, K, device=dev, generator=g))     # some channels larger than others
        s["x"] = x.to(torch.bfloat16)
        i32 = dict(dtype=torch.int32, device=dev)
        s["row_of"] = torch.empty(T, k, **i32)
        if c["form"] == "masked":
            m = c["max_m"]
            s["masked_m"] = torch.empty(G, **i32)
            s["slot_of"] = torch.empty(G, m, **i32)
            s["a"] = torch.zeros(G, m, K, dtype=torch.uint8, device=dev)
            s["sfa"] = torch.zeros(G, K // BLOCK, m, device=dev)
        else:
            M = _bound_rows(c)
            s["counts"] = torch.empty(G, **i32)
            s["slot_of"] = torch.empty(M, **i32)
            s["layout"] = torch.empty(M, **i32)
            s["a"] = torch.zeros(M, K, dtype=torch.uint8, device=dev)
            s["sfa"] = torch.zeros(M // BLOCK if c["form"] == "kgrouped" else K // BLOCK,
                                   K if c["form"] == "kgrouped" else M, device=dev)
            if c["form"] == "kgrouped":        # the maps are the forward pass's
                s["layout"], s["row_of"], s["slot_of"], s["counts"] = _layout_plain(s)
        return s
    if c["op"] == "rows_back":
        N = c["N"]
        s["c"] = dict(c, groups=experts, first=0, form="contiguous")
        M = _bound_rows(s["c"])
        i32 = dict(dtype=torch.int32, device=dev)
        s["slot_of"], s["layout"], s["counts"] = torch.empty(M, **i32), torch.empty(M, **i32), torch.empty(experts, **i32)
        s["row_of"] = _layout_plain(s)[1].contiguous()
        s["row_of"].masked_fill_(torch.rand(T, k, device=dev, generator=g) < 0.05, -1)
        s["rows"] = torch.randn(M, N, device=dev, generator=g, dtype=torch.bfloat16)
        s["residual"] = torch.randn(T, N, device=dev, generator=g, dtype=torch.bfloat16) if c["residual"] else None
        s["d"] = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
        if c["direction"] == "weight_grad":
            s["grad_d"] = torch.randn(T, N, device=dev, generator=g, dtype=torch.bfloat16)
            s["grad_weights"] = torch.empty(T, k, device=dev)
        return s
    K, N, R, L = c["K"], c["N"], c["R"], c["adapters"]
    s["x"] = torch.randn(T, K, device=dev, generator=g, dtype=torch.bfloat16)
    s["a"] = (torch.randn(L, R, K, device=dev, generator=g) * K ** -0.5).to(torch.bfloat16)
    s["b"] = (torch.randn(L, N, R, device=dev, generator=g) * 0.1).to(torch.bfloat16)
    s["scales"] = 0.5 + torch.rand(L, device=dev, generator=g)
    n = -(-T // c["runs"])
    ids = torch.randint(0, L, (n,), device=dev, generator=g, dtype=torch.int32).repeat_interleave(c["runs"])[:T]
    idle = (torch.rand(n, device=dev, generator=g) < c["idle"]).repeat_interleave(c["runs"])[:T]
    s["adapter_ids"] = ids.masked_fill(idle, -1).contiguous()
    s["base"] = torch.randn(T, N, device=dev, generator=g, dtype=torch.bfloat16) if c["residual"] else None
    s["d"] = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _scores_plain(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _route_plain(s):
    c = s["c"]
    x = s["logits"].float()
    T, E, G = c["T"], c["E"], c["num_groups"]
    p = _scores_plain(x, c["score"])
    key = p if s["bias"] is None else p + s["bias"]
    key = key.masked_fill(x == -math.inf, -math.inf)
    if G > 1:
        per = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        gs = per.masked_fill(per == -math.inf, 0.0).sum(2).masked_fill(per[:, :, 0] == -math.inf, -math.inf)
        kept = gs.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = key.masked_fill(~mask.repeat_interleave(E // G, 1), -math.inf)
    order = key.sort(dim=1, descending=True, stable=True)
    took = order.values[:, :c["top_k"]] != -math.inf
    ids = order.indices[:, :c["top_k"]]
    w = p.gather(1, ids).masked_fill(~took, 0.0)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return ids.to(torch.int32).masked_fill(~took, -1), w * c["scale"]


def _route_backward_plain(s):
    c = s["c"]
    x = s["logits"].float()
    p = _scores_plain(x, c["score"])
    took = s["ids"] >= 0
    at = s["ids"].clamp_min(0).long()
    w = p.gather(1, at).masked_fill(~took, 0.0)
    gw = s["grad_weights"].masked_fill(~took, 0.0) * c["scale"]
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        gw = (gw - (gw * w).sum(1, keepdim=True) / total) / total
    gp = torch.zeros_like(p).scatter_add_(1, at, gw.masked_fill(~took, 0.0))
    if c["score"] == "sigmoid":
        gx = gp * p * (1.0 - p)
    else:
        gx = p * (gp - (gp * p).sum(1, keepdim=True))
    return gx.to(s["logits"].dtype)


def _layout_plain(s):
    """(layout or masked_m, row_of, slot_of, counts) of the tokens' choices."""
    c = s["c"]
    G = c["groups"]
    local = s["ids"].view(-1).long() - c["first"]
    dev = local.device
    group = torch.where((local >= 0) & (local < G), local, torch.full_like(local, G))
    counts = torch.zeros(G + 1, dtype=torch.long, device=dev).scatter_add_(0, group, torch.ones_like(group))
    order = group.sort(stable=True).indices
    first = counts.cumsum(0) - counts
    rank = torch.empty_like(group)
    rank[order] = torch.arange(group.numel(), device=dev) - first[group[order]]
    if c["form"] == "masked":
        m = c["max_m"]
        row = torch.where((group < G) & (rank < m), group * m + rank, torch.full_like(group, -1))
        rows = G * m
    else:
        rows = s["slot_of"].numel()
        span = (counts[:G] + BLOCK - 1) // BLOCK * BLOCK
        start = torch.cat([span.cumsum(0) - span, torch.zeros(1, dtype=torch.long, device=dev)])
        row = start[group] + rank
        row = torch.where((group < G) & (row < rows), row, torch.full_like(row, -1))
    live = row >= 0
    slot = torch.full((rows + 1,), -1, dtype=torch.long, device=dev)
    slot[torch.where(live, row, torch.full_like(row, rows))] = torch.arange(group.numel(), device=dev)
    slot = slot[:rows]
    i32 = torch.int32
    row_of = row.to(i32).view(c["T"], c["top_k"])
    if c["form"] == "masked":
        return counts[:G].clamp_max(c["max_m"]).to(i32), row_of, slot.to(i32).view(G, -1), counts[:G].to(i32)
    layout = torch.where(slot >= 0, group[slot.clamp_min(0)], torch.full_like(slot, -1))
    return layout.to(i32), row_of, slot.to(i32), counts[:G].to(i32)


def _scale_plain(amax, pow2):
    sf = amax.clamp_min(TINY) / E4M3_MAX
    if pow2:
        m, e = torch.frexp(sf)
        sf = torch.ldexp(torch.ones_like(sf), torch.where(m == 0.5, e - 1, e))
    return torch.where(amax > 0, sf, torch.ones_like(sf))


def _rows_out_plain(s):
    c = s["c"]
    K, k = c["K"], c["top_k"]
    if c["form"] == "kgrouped":
        slot = s["slot_of"].long()
        x = s["x"][slot.clamp_min(0) // k].float()
        if c["weighted"]:
            x = x * s["weights"].view(-1)[slot.clamp_min(0)].unsqueeze(1)
        x = x.masked_fill((slot < 0).unsqueeze(1), 0.0).view(-1, BLOCK, K)
        sf = _scale_plain(x.abs().amax(1), c["pow2"])
        q = (x * (1.0 / sf).unsqueeze(1)).clamp(-E4M3_MAX, E4M3_MAX)
        return {"a": q.to(torch.float8_e4m3fn).view(-1, K), "sfa": sf}
    first, row_of, slot_of, counts = _layout_plain(s)
    slot = slot_of.view(-1).long()
    rows = (slot >= 0).nonzero().view(-1)
    took = slot[rows]
    x = s["x"][took // k].float()
    if c["weighted"]:
        x = x * s["weights"].view(-1)[took].unsqueeze(1)
    x = x.view(-1, K // BLOCK, BLOCK)
    sf = _scale_plain(x.abs().amax(2), c["pow2"])
    q = (x * (1.0 / sf).unsqueeze(2)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    s["a"].view(-1, K)[rows] = q.view(torch.uint8).view(-1, K)
    if c["form"] == "masked":
        m = c["max_m"]
        s["sfa"][rows // m, :, rows % m] = sf
    else:
        s["sfa"][:, rows] = sf.t()
    out = {"a": s["a"].view(torch.float8_e4m3fn), "sfa": s["sfa"], "row_of": row_of, "slot_of": slot_of}
    out["masked_m" if c["form"] == "masked" else "layout"] = first
    if c["form"] != "masked":
        out["counts"] = counts
    return out


def _rows_back_plain(s):
    c = s["c"]
    at = s["row_of"].long()
    live = at >= 0
    r = s["rows"][at.clamp_min(0)].float().masked_fill(~live.unsqueeze(2), 0.0)
    if c["direction"] == "weight_grad":
        return (r * s["grad_d"].float().unsqueeze(1)).sum(2)
    if c["weighted"]:
        r = r * s["weights"].unsqueeze(2)
    d = r.sum(1)
    if c["residual"]:
        d = d + s["residual"].float()
    return d.to(torch.bfloat16)


def _lora_plain(s):
    c = s["c"]
    T, L, R = c["T"], c["adapters"], c["R"]
    ids = s["adapter_ids"].long()
    h = (s["x"].float() @ s["a"].view(L * R, -1).float().t()).view(T, L, R)
    mine = ids.unsqueeze(1) == torch.arange(L, device=ids.device)
    h = torch.where(mine.unsqueeze(2), h * s["scales"].view(1, L, 1), torch.zeros_like(h)).view(T, L * R)
    d = h @ s["b"].float().transpose(1, 2).reshape(L * R, -1)
    if c["residual"]:
        d = d + s["base"].float()
    return d.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    s, c = state, state["c"]
    if c["op"] == "route":
        if c["direction"] == "backward":
            if not own:
                return _route_backward_plain(s)
            _dg().dg_route_topk_backward(s["logits"], s["ids"], s["grad_weights"], s["grad_logits"], score=c["score"],
                                         renormalize=c["renormalize"], scale=c["scale"])
            return s["grad_logits"]
        if not own:
            return _route_plain(s)
        _dg().dg_route_topk(s["logits"], s["bias"], s["ids"], s["weights"], score=c["score"],
                            num_groups=c["num_groups"], topk_groups=c["topk_groups"], group_top=c["group_top"],
                            renormalize=c["renormalize"], scale=c["scale"])
        return s["ids"], s["weights"]
    if c["op"] == "rows_out":
        if not own:
            return _rows_out_plain(s)
        dg = _dg()
        a = s["a"].view(torch.float8_e4m3fn)
        if c["form"] == "kgrouped":
            dg.dg_k_grouped_scatter_fp8(s["x"], s["weights"], s["slot_of"], c["top_k"], a, s["sfa"],
                                        pow2_scales=c["pow2"])
            return {"a": a, "sfa": s["sfa"]}
        if c["form"] == "masked":
            dg.dg_m_grouped_layout_masked(s["ids"], c["first"], s["masked_m"], s["row_of"], s["slot_of"])
            dg.dg_m_grouped_scatter_fp8_masked(s["x"], s["weights"], s["row_of"], s["slot_of"], a, s["sfa"],
                                               pow2_scales=c["pow2"])
            return {"a": a, "sfa": s["sfa"], "row_of": s["row_of"], "slot_of": s["slot_of"], "masked_m": s["masked_m"]}
        dg.dg_m_grouped_layout_contiguous(s["ids"], c["first"], s["layout"], s["row_of"], s["slot_of"], s["counts"])
        dg.dg_m_grouped_scatter_fp8_contiguous(s["x"], s["weights"], s["row_of"], s["slot_of"], a, s["sfa"],
                                               pow2_scales=c["pow2"])
        return {"a": a, "sfa": s["sfa"], "row_of": s["row_of"], "slot_of": s["slot_of"], "layout": s["layout"],
                "counts": s["counts"]}
    if c["op"] == "rows_back":
        if not own:
            return _rows_back_plain(s)
        if c["direction"] == "weight_grad":
            _dg().dg_m_grouped_gather_weight_grad(s["rows"], s["row_of"], s["grad_d"], s["grad_weights"])
            return s["grad_weights"]
        _dg().dg_m_grouped_gather(s["rows"], s["row_of"], s["weights"], s["residual"], s["d"])
        return s["d"]
    if not own:
        return _lora_plain(s)
    _dg().dg_lora_bf16_nt(s["x"], s["a"], s["b"], s["scales"], s["adapter_ids"], s["base"], s["d"])
    return s["d"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _route_exact(s):
    c = s["c"]
    x = s["logits"].double()
    back = c["direction"] == "backward"
    if c["score"] == "sigmoid":
        logp = -torch.nn.functional.softplus(-x)
    else:
        logp = x - torch.logsumexp(x, 1, keepdim=True)
    p = logp.exp().nan_to_num(nan=0.0)
    if back:
        ids = s["ids"].long()
    else:
        key = (p if s["bias"] is None else p + s["bias"].double()).masked_fill(x == -math.inf, -math.inf)
        per = c["E"] // c["num_groups"]
        if c["num_groups"] > 1:
            of_group = key.view(c["T"], -1, per)
            some = of_group.amax(2) > -math.inf
            best = of_group.topk(min(per, c["group_top"]), 2).values
            best = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
            best = torch.where(some, best, torch.full_like(best, -math.inf))
            rank = best.argsort(dim=1, descending=True, stable=True).argsort(1)
            key = torch.where((rank < c["topk_groups"]).repeat_interleave(per, 1), key, torch.full_like(key, -math.inf))
        ids = key.argsort(dim=1, descending=True, stable=True)[:, :c["top_k"]]
        ids = torch.where(key.gather(1, ids) > -math.inf, ids, torch.full_like(ids, -1))
    has = (ids >= 0).double()
    chosen = p.gather(1, ids.clamp_min(0)) * has
    z = chosen.sum(1, keepdim=True)
    z = torch.where(z > 0, z, torch.ones_like(z))
    w = chosen / z if c["renormalize"] else chosen
    if not back:
        return None, w * c["scale"]
    g = s["grad_weights"].double() * has * c["scale"]
    u = g * w                                        # dL/dlog(score) of the chosen, before the normalisations
    if c["renormalize"]:
        u = u - w * u.sum(1, keepdim=True)
    out = torch.zeros_like(p)
    if c["score"] == "sigmoid":
        out.scatter_add_(1, ids.clamp_min(0), u * has * (1 - chosen))
    else:
        out.scatter_add_(1, ids.clamp_min(0), u * has)
        out -= p * (u * has).sum(1, keepdim=True)
    return out


def _e4m3_exact(v):
    """v rounded to the nearest e4m3 value, ties to even."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    e = torch.frexp(v).exponent.clamp_min(-5) - 4    # the exponent of the last place
    step = torch.ldexp(torch.ones_like(v), e)
    return torch.round(v / step) * step


def _rows_out_exact(s):
    c = s["c"]
    K, k = c["K"], c["top_k"]
    x, w = s["x"].double(), s["weights"]
    first, row_of, slot_of, _ = _layout_plain(s) if c["form"] != "kgrouped" else (None, None, s["slot_of"], None)
    slot = slot_of.reshape(-1).long()

    def quantised(v, dim):
        amax = v.abs().amax(dim, keepdim=True)
        sf = amax.clamp_min(TINY) / E4M3_MAX
        if c["pow2"]:
            sf = torch.exp2(torch.ceil(torch.log2(sf.float().double())))
        sf = torch.where(amax > 0, sf, torch.ones_like(sf))
        return _e4m3_exact(v / sf), sf

    a = torch.zeros(slot.numel(), K, dtype=torch.float32, device=x.device)
    masked = c["form"] == "masked"
    sfa = torch.zeros(s["sfa"].shape, dtype=torch.double, device=x.device)
    step = 8192
    for r in range(0, slot.numel(), step):           # 64-bit copies of a few rows at a time
        t = slot[r:r + step]
        v = x[t.clamp_min(0) // k]
        if w is not None:
            v = v * w.double().view(-1)[t.clamp_min(0)].unsqueeze(1)
        live = (t >= 0).unsqueeze(1)
        v = torch.where(live, v, torch.zeros_like(v))
        n = t.numel()
        if c["form"] == "kgrouped":
            q, sf = quantised(v.view(n // BLOCK, BLOCK, K), 1)
            sfa[r // BLOCK:(r + n) // BLOCK] = sf.squeeze(1)
            a[r:r + n] = q.view(n, K).float()
            continue
        q, sf = quantised(v.view(n, K // BLOCK, BLOCK), 2)
        a[r:r + n] = q.view(n, K).float()
        sf = torch.where(live, sf.squeeze(2), torch.zeros_like(sf.squeeze(2)))
        if masked:
            at = torch.arange(r, r + n, device=x.device)
            sfa[at // c["max_m"], :, at % c["max_m"]] = sf
        else:
            sfa[:, r:r + n] = sf.t()
    a = a.view(s["a"].shape)
    if c["form"] == "kgrouped":
        return {"a": a, "sfa": sfa}
    out = {"a": a, "sfa": sfa, "row_of": None, "slot_of": None}
    if masked:
        out["masked_m"] = None
    else:
        out["layout"], out["counts"] = None, None
    return out


def _rows_back_exact(s):
    c = s["c"]
    T, N = c["T"], c["N"]
    back = c["direction"] == "weight_grad"
    out = torch.zeros(T, c["top_k"] if back else N, dtype=torch.double, device=s["rows"].device)
    if not back and c["residual"]:
        out += s["residual"].double()
    for j in range(c["top_k"]):
        at = s["row_of"][:, j].long()
        tokens = (at >= 0).nonzero().view(-1)
        rows = s["rows"][at[tokens]].double()
        if back:
            out[tokens, j] = (rows * s["grad_d"][tokens].double()).sum(1)
        else:
            out[tokens] += rows * s["weights"][tokens, j].double().unsqueeze(1) if c["weighted"] else rows
    return out


def _lora_exact(s):
    c = s["c"]
    out = torch.zeros(c["T"], c["N"], dtype=torch.double, device=s["x"].device)
    if c["residual"]:
        out += s["base"].double()
    for i in range(c["adapters"]):
        tokens = (s["adapter_ids"] == i).nonzero().view(-1)
        if tokens.numel():
            h = s["x"][tokens].double() @ s["a"][i].double().t()
            out[tokens] += s["scales"][i].double() * (h @ s["b"][i].double().t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _route_exact, "rows_out": _rows_out_exact, "rows_back": _rows_back_exact,
            "lora": _lora_exact}[case["op"]](s)
