"""More operators of a mixture-of-experts layer, as measured.

Three operators, each with its plain form in elementary torch operations and the
calls a user makes of this package:

  balance    the router's balance loss per sequence with the experts' counts, and
             its gradient, added to the routing weights' own
  gemv       products of a few tokens with 4-bit weights (E2M1 with a power-of-two
             scale per 32 values, or integers with group scales and zero points):
             a dense projection, or the experts of every choice
  clip       the norm of all gradients together, and the gradients scaled to it

``own`` false: plain torch, computed in 32 bits and rounded once at the end.
``own`` true: the package's kernels."""
import math

import torch

own = False

BLOCK = 128           # K values per word of four E8M0 exponents
TINY_NORM = 1e-6      # added to the norm before the division, as training code does


def _dg():
    import moe_grouped_gemm_nt_amd as dg
    return dg


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _balance(direction, T, E, top_k, score, seqs=1, dtype="float32", masked=0.0, onto=False, tail=0.0):
    return dict(op="balance", direction=direction, T=T, E=E, top_k=top_k, score=score, seqs=seqs, dtype=dtype,
                masked=masked, onto=onto, tail=tail)


def _gemv(form, M, N, K, group=32, scales="float32", zeros=False, residual=False, wide=0):
    """wide: elements by which the rows of x lie further apart than K."""
    return dict(op="gemv", form=form, M=M, N=N, K=K, group=group, scales=scales, zeros=zeros, residual=residual,
                wide=wide, top_k=0, experts=1, first=0, groups=1, per_choice=False)


def _experts(form, T, top_k, experts, first, groups, N, K, group=32, scales="float32", zeros=False, per_choice=False,
             residual=False):
    return dict(op="gemv", form=form, M=T, N=N, K=K, group=group, scales=scales, zeros=zeros, residual=residual,
                wide=0, top_k=top_k, experts=experts, first=first, groups=groups, per_choice=per_choice)


def _clip(tensors, smallest, largest, halves, big=0):
    """tensors: how many, of smallest to largest values, a share `halves` of them bf16; big: values of one more in fp32."""
    return dict(op="clip", tensors=tensors, smallest=smallest, largest=largest, halves=halves, big=big)


def listed():
    return [
        # a micro-batch of 512 tokens of a small router: a few microseconds, all latency
        dict(_balance("forward", 512, 64, 6, "softmax"), name="balance_small"),
        # a training batch of 8 sequences of their own lengths, 256 experts, 8 chosen, and some padding behind the last
        dict(_balance("forward", 16384, 256, 8, "sigmoid", seqs=8, tail=0.02), name="balance_sequences"),
        # the gradient onto the routing gradient: a batch of odd length, an expert count that is no power of two, bf16
        dict(_balance("backward", 20479, 60, 4, "softmax", dtype="bfloat16", masked=0.02, onto=True),
             name="balance_backward_softmax"),
        # the gradient of the batch of sequences
        dict(_balance("backward", 16384, 256, 8, "sigmoid", seqs=8, onto=True, tail=0.02),
             name="balance_backward_sequences"),
        # decoding one request: the decode projection, 2112 x 7168, onto a residual
        dict(_gemv("fp4", 1, 2112, 7168, residual=True), name="gemv_one_token"),
        # decoding 64 requests: a 4096 x 7168 projection
        dict(_gemv("fp4", 64, 4096, 7168), name="gemv_batch"),
        # speculative decoding: 5 tokens through a 7168 x 16384 projection of integers with zero points, x a column slice
        dict(_gemv("int4", 5, 7168, 16384, group=128, scales="bfloat16", zeros=True, wide=128), name="gemv_int4"),
        # decoding 64 requests over 4 GPUs: the 32 experts of 128 that are here, up to 4096 x 7168 each
        dict(_experts("fp4", 64, 8, 128, 32, 32, 4096, 7168), name="experts_batch"),
        # one request's way down: its 8 experts, each on its own row, an odd number of columns
        dict(_experts("int4", 1, 8, 16, 0, 16, 7165, 2048, group=64, scales="float32", per_choice=True),
             name="experts_one_token"),
        # the gradients of a small layer: biases, norms and small matrices, all latency
        dict(_clip(47, 1, 40000, 0.5), name="clip_small"),
        # the gradients of a dense layer in bf16 and fp32
        dict(_clip(31, 100, 9000000, 0.7), name="clip_layer"),
        # the weight gradients of 8 experts of 4096 x 7168 in fp32, as the K-grouped product leaves them, and the rest
        dict(_clip(13, 64, 2000000, 0.3, big=8 * 4096 * 7168), name="clip_experts"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, mostly odd."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n if n < 4 or rng.random() < 0.25 and n % 1024 else n | 1))


_KS = [128, 256, 384, 640, 896, 1024, 1408, 2048, 4096, 4224, 7168, 8192, 16384]
_NS = [1, 24, 100, 129, 513, 1000, 2047, 2112, 4096, 7165, 7168, 7424, 16384]


def _drawn(rng):
    op = rng.choice(["balance", "balance", "gemv", "gemv", "gemv", "experts", "experts", "clip"])
    if op == "balance":
        E = rng.choice([8, 16, 48, 60, 64, 96, 128, 160, 256, 320, 384, 512])
        return _balance(rng.choice(["forward", "backward"]), _log_int(rng, 1, 32768), E,
                        min(E // 2, rng.choice([1, 2, 4, 6, 8, 10])), rng.choice(["softmax", "sigmoid"]),
                        seqs=rng.choice([1, 1, 2, 7, 32, 200]), dtype=rng.choice(["float32", "bfloat16"]),
                        masked=rng.choice([0.0, 0.0, 0.05]), onto=rng.random() < 0.5,
                        tail=rng.choice([0.0, 0.0, 0.1]))
    if op == "clip":
        return _clip(_log_int(rng, 1, 60), 1, _log_int(rng, 1000, 20000000), rng.choice([0.0, 0.5, 1.0]))
    form = rng.choice(["fp4", "int4"])
    more = dict(residual=rng.random() < 0.4)
    if form == "int4":
        more.update(group=rng.choice([32, 64, 128]), scales=rng.choice(["float32", "bfloat16"]),
                    zeros=rng.random() < 0.5)
    if op == "gemv":
        return _gemv(form, _log_int(rng, 1, 64), rng.choice(_NS), rng.choice(_KS), wide=rng.choice([0, 0, 8, 256]),
                     **more)
    groups = rng.choice([1, 3, 8, 16, 31, 32, 64])
    share = rng.choice([1, 1, 2, 4])
    return _experts(form, _log_int(rng, 1, 64), min(rng.choice([1, 2, 4, 6, 8]), groups * share), groups * share,
                    groups * rng.randrange(share), groups, rng.choice(_NS), rng.choice(_KS),
                    per_choice=rng.random() < 0.4, **more)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        c = _drawn(rng)
        if _cost(c) <= most[c["op"]]:
            return c


def _cost(c):
    """Bytes of a case's pass, with all weights that it holds."""
    if c["op"] == "gemv":
        return c["groups"] * c["N"] * c["K"] + c["M"] * max(1, c["top_k"]) * c["N"]
    return work(c)["bytes"]


def _sizes(c):
    """The tensors' sizes, spread over their logarithm: the same for every seed."""
    n, lo, hi = c["tensors"], c["smallest"], c["largest"]
    sizes = [int(lo * (hi / lo) ** (i / max(1, n - 1))) | 1 for i in range(n)]
    return [min(hi, s) for s in sizes]


def _is_half(c, i):
    return (i * 7919 % 100) < 100 * c["halves"]


def work(c):
    if c["op"] == "balance":
        T, E = c["T"], c["E"]
        size = 4 if c["dtype"] == "float32" else 2
        if c["direction"] == "forward":
            return {"bytes": T * (E * size + c["top_k"] * 4) + c["seqs"] * (E * 4 + 4), "flops": 6 * T * E}
        return {"bytes": T * E * size * (3 if c["onto"] else 2) + c["seqs"] * (E * 4 + 4), "flops": 10 * T * E}
    if c["op"] == "clip":
        n = sum(s * (2 if _is_half(c, i) else 4) for i, s in enumerate(_sizes(c))) + c["big"] * 4
        values = sum(_sizes(c)) + c["big"]
        return {"bytes": 2 * n + 4, "flops": 3 * values}
    M, N, K = c["M"], c["N"], c["K"]
    if c["form"] == "fp4":
        per_expert = N * K / 2 + N * K / 32
    else:
        per_expert = N * K / 2 + N * K / c["group"] * ((4 if c["scales"] == "float32" else 2) + (1 if c["zeros"] else 0))
    if not c["top_k"]:
        return {"bytes": per_expert + M * K * 2 + M * N * 2 * (2 if c["residual"] else 1), "flops": 2 * M * N * K}
    n = M * c["top_k"]
    here = n * c["groups"] / c["experts"]
    used = c["groups"] * (1 - (1 - c["top_k"] / c["experts"]) ** M)        # experts that some choice has
    rows = here if c["per_choice"] else M * (1 - (1 - c["groups"] / c["experts"]) ** c["top_k"])
    return {"bytes": used * per_expert + rows * K * 2 + n * N * 2 * (2 if c["residual"] else 1) + n * 4,
            "flops": 2 * here * N * K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _choices(g, T, experts, top_k, dev):
    """Expert ids [T][top_k] without repeats, some experts liked more than others."""
    liking = torch.randn(experts, device=dev, generator=g) * 0.5
    noise = torch.rand(T, experts, device=dev, generator=g).clamp_(1e-7, 1 - 1e-7)
    return (liking - torch.log(-torch.log(noise))).topk(top_k, 1).indices.to(torch.int32)


def _seq_of(starts, T):
    """Each token's sequence, or the number of sequences for those behind the last."""
    return torch.searchsorted(starts[1:].contiguous(), torch.arange(T, dtype=torch.int32, device=starts.device),
                              right=True)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "balance":
        T, E, S, k = c["T"], c["E"], c["seqs"], c["top_k"]
        dtype = getattr(torch, c["dtype"])
        x = torch.randn(T, E, device=dev, generator=g) * 1.5 + torch.randn(E, device=dev, generator=g) * 0.5
        if c["masked"]:
            x.masked_fill_(torch.rand(T, E, device=dev, generator=g) < c["masked"], -math.inf)
            x[T // 2] = -math.inf                                # a token that no expert may take
        s["logits"] = x.to(dtype)
        s["ids"] = x.topk(k, 1).indices.to(torch.int32)
        s["ids"][T // 3, k - 1] = -1                             # a choice that was dropped
        last = T - int(T * c["tail"])
        cuts = torch.sort(torch.randint(0, last + 1, (S - 1,), device=dev, generator=g)).values
        ends = torch.tensor([0, last], device=dev)
        s["starts"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
        s["loss"] = torch.empty(S, device=dev)
        s["counts"] = torch.empty(S, E, dtype=torch.int32, device=dev)
        if c["direction"] == "backward":
            s["counts"] = _counts_plain(s)
            s["grad_loss"] = 0.01 * (1 + torch.rand(S, device=dev, generator=g)) * max(1, T // S)
            s["onto"] = (torch.randn(T, E, device=dev, generator=g) * 0.003).to(dtype) if c["onto"] else None
            s["grad_logits"] = torch.empty_like(s["logits"])
        return s
    if c["op"] == "clip":
        sizes = _sizes(c)
        for kind, dtype in (("f", torch.float32), ("h", torch.bfloat16)):
            mine = [n for i, n in enumerate(sizes) if _is_half(c, i) == (kind == "h")]
            total = sum(mine) + (c["big"] if kind == "f" else 0)
            flat = torch.randn(total, device=dev, generator=g) * 0.02
            s[kind] = flat.to(dtype)                             # gradients lie one behind the other, as in a bucket
            s["out_" + kind] = torch.empty_like(s[kind])
            mine += [c["big"]] if kind == "f" and c["big"] else []
            s["grads_" + kind] = list(s[kind].split(mine)) if mine else []
            s["outs_" + kind] = list(s["out_" + kind].split(mine)) if mine else []
        s["grads"], s["outs"] = s["grads_f"] + s["grads_h"], s["outs_f"] + s["outs_h"]
        s["norm"] = torch.empty(1, device=dev)
        s["max_norm"] = 0.5
        return s
    M, N, K, G = c["M"], c["N"], c["K"], c["groups"]
    k = c["top_k"]
    rows = M * k if c["per_choice"] else M
    x = torch.randn(rows, K + c["wide"], device=dev, generator=g)
    x *= torch.exp(0.5 * torch.randn(1, K + c["wide"], device=dev, generator=g))        # some channels larger than others
    s["x"] = x.to(torch.bfloat16)[:, :K]
    lead = (G,) if k else ()
    s["b"] = torch.randint(0, 256, (*lead, N, K // 2), device=dev, generator=g, dtype=torch.uint8)
    if c["form"] == "fp4":
        e = torch.randint(-3, 2, (*lead, K // BLOCK, N, 4), device=dev, generator=g) + 127 - int(math.log2(K) / 2)
        s["sfb"] = e.to(torch.uint8).view(torch.int32).view(*lead, K // BLOCK, N)
    else:
        sc = (0.5 + torch.rand(*lead, K // c["group"], N, device=dev, generator=g)) * 0.2 * K ** -0.5
        s["scales"] = sc.to(getattr(torch, c["scales"]))
        s["zeros"] = None
        if c["zeros"]:
            s["zeros"] = torch.randint(5, 12, sc.shape, device=dev, generator=g, dtype=torch.uint8)
    n = M * k if k else M
    if k:
        s["ids"] = _choices(g, M, c["experts"], k, dev)
    s["base"] = torch.randn(n, N, device=dev, generator=g, dtype=torch.bfloat16) if c["residual"] else None
    s["d"] = torch.empty(n, N, dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _shares_plain(x, score):
    """(each token's shares of the experts, what a share's gradient has besides): 0 for masked experts."""
    masked = x == -math.inf
    top = x.amax(1, keepdim=True).nan_to_num(neginf=0.0)
    if score == "softmax":
        e, rest = torch.exp(x - top), None
    else:
        e, rest = 1.0 / (1.0 + torch.exp(-x)), 1.0 / (1.0 + torch.exp(x))
    e = e.masked_fill(masked, 0.0)
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total)), rest


def _members(s):
    """[sequences][tokens], 1.0 where the token is of that sequence."""
    c = s["c"]
    seq = _seq_of(s["starts"], c["T"])
    return (seq.unsqueeze(0) == torch.arange(c["seqs"], device=seq.device).unsqueeze(1)).float()


def _counts_plain(s):
    c = s["c"]
    E = c["E"]
    ids = s["ids"].long()
    at = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E))
    chosen = torch.zeros(c["T"], E + 1, device=ids.device).scatter_add_(1, at, torch.ones_like(at, dtype=torch.float32))
    return (_members(s) @ chosen[:, :E]).to(torch.int32)


def _balance_plain(s):
    c = s["c"]
    E = c["E"]
    p, rest = _shares_plain(s["logits"].float(), c["score"])
    n = (s["starts"][1:] - s["starts"][:-1]).float()
    weight = E / (c["top_k"] * n.clamp_min(1) ** 2)              # [S]
    if c["direction"] == "forward":
        counts = _counts_plain(s)
        return weight * (counts * (_members(s) @ p)).sum(1), counts
    seq = _seq_of(s["starts"], c["T"])
    zero = torch.zeros(1, device=p.device)
    weight = torch.cat([weight * s["grad_loss"], zero])[seq].view(-1, 1)
    counts = torch.cat([s["counts"].float(), torch.zeros(1, E, device=p.device)])[seq]
    gx = weight * p * (counts - (p * counts).sum(1, keepdim=True))
    if rest is not None:
        gx = (gx * rest).masked_fill(s["logits"] == -math.inf, 0.0)
    if s["onto"] is not None:
        gx = gx + s["onto"].float()
    return gx.to(s["logits"].dtype)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _weights_plain(s):
    """The weights [groups * N][K] in fp32."""
    c = s["c"]
    N, K, G = c["N"], c["K"], c["groups"]
    b = s["b"].view(G, N, K // 2)
    if c["form"] == "fp4":
        v = torch.tensor(_E2M1, device=b.device)
        pairs = torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)        # a byte's two values, the low one first
        w = pairs[b.int()].view(G, N, K // 32, 32)
        e = s["sfb"].view(torch.uint8).view(G, K // BLOCK, N, 4).permute(0, 2, 1, 3).reshape(G, N, K // 32, 1)
        return (w * torch.exp2(e.float() - 127.0)).view(G * N, K)
    g = c["group"]
    w = torch.stack([b & 15, b >> 4], 3).float().view(G, N, K // g, g)
    zero = 8.0
    if s["zeros"] is not None:
        zero = s["zeros"].view(G, K // g, N).transpose(1, 2).float().unsqueeze(3)
    sc = s["scales"].view(G, K // g, N).transpose(1, 2).float().unsqueeze(3)
    return ((w - zero) * sc).view(G * N, K)


def _gemv_plain(s):
    c = s["c"]
    N, G, k = c["N"], c["groups"], c["top_k"]
    d = s["x"].float() @ _weights_plain(s).t()
    if k:
        d = d.view(-1, G, N)                                     # every row of x through every expert
        at = s["ids"].view(-1).long() - c["first"]
        here = (at >= 0) & (at < G)
        row = torch.arange(at.numel(), device=at.device) // (1 if c["per_choice"] else k)
        d = d[row, at.clamp(0, G - 1)].masked_fill(~here.unsqueeze(1), 0.0)
    if s["base"] is not None:
        d = d + s["base"].float()
    return d.to(torch.bfloat16)


def _clip_plain(s):
    total = torch.stack([g.double().square().sum() if g.numel() > 1 << 24 else g.float().square().sum().double()
                         for g in s["grads"]]).sum()
    norm = total.sqrt().float()
    factor = (s["max_norm"] / (norm + TINY_NORM)).clamp_max(1.0)
    outs = [o.copy_(g.float() * factor) for g, o in zip(s["grads"], s["outs"])]
    assert len(outs) == len(s["grads"])
    return {"norm": norm.view(1), "f": s["out_f"], "h": s["out_h"]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    s, c = state, state["c"]
    if c["op"] == "balance":
        if not own:
            return _balance_plain(s)
        if c["direction"] == "forward":
            _dg().dg_route_balance(s["logits"], s["ids"], s["starts"], s["loss"], s["counts"], score=c["score"])
            return s["loss"], s["counts"]
        _dg().dg_route_balance_backward(s["logits"], s["counts"], s["starts"], s["grad_loss"], s["onto"],
                                        s["grad_logits"], c["top_k"], score=c["score"])
        return s["grad_logits"]
    if c["op"] == "clip":
        if not own:
            return _clip_plain(s)
        dg = _dg()
        dg.dg_grad_norm(s["grads"], s["norm"])
        dg.dg_grad_clip(s["grads"], s["outs"], s["norm"], s["max_norm"])
        return {"norm": s["norm"], "f": s["out_f"], "h": s["out_h"]}
    if not own:
        return _gemv_plain(s)
    dg = _dg()
    if c["top_k"]:
        if c["form"] == "fp4":
            dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(s["x"], s["ids"], c["first"], s["b"], s["sfb"], s["base"], s["d"])
        else:
            dg.dg_m_grouped_bf16_int4_gemv_nt_topk(s["x"], s["ids"], c["first"], s["b"], s["scales"], s["zeros"],
                                                   s["base"], s["d"])
    elif c["form"] == "fp4":
        dg.dg_bf16_fp4_gemv_nt(s["x"], s["b"], s["sfb"], s["base"], s["d"])
    else:
        dg.dg_bf16_int4_gemv_nt(s["x"], s["b"], s["scales"], s["zeros"], s["base"], s["d"])
    return s["d"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _balance_exact(s):
    c = s["c"]
    T, E, S, k = c["T"], c["E"], c["seqs"], c["top_k"]
    starts = s["starts"].tolist()
    back = c["direction"] == "backward"
    x = s["logits"].double().requires_grad_(back)
    allowed = torch.isfinite(s["logits"])
    losses = []
    for q in range(S):
        a, b = starts[q], starts[q + 1]
        if a == b:
            losses.append(torch.zeros((), dtype=torch.double, device=x.device))
            continue
        rows, ok = x[a:b], allowed[a:b]
        safe = torch.where(ok, rows, torch.zeros_like(rows))
        logs = safe if c["score"] == "softmax" else torch.nn.functional.logsigmoid(safe)
        logs = torch.where(ok, logs, torch.full_like(logs, -1e300))
        share = torch.softmax(logs, 1) * ok                      # sigmoid / sum of sigmoids = softmax of their logarithms
        if back:
            f = s["counts"][q].double()
        else:
            ids = s["ids"][a:b]
            f = torch.bincount(ids[ids >= 0], minlength=E).double()
        f = f * E / (k * (b - a))
        losses.append((f * share.mean(0)).sum())
    losses = torch.stack(losses)
    if not back:
        return losses, None
    (losses * s["grad_loss"].double()).sum().backward()
    return x.grad + (s["onto"].double() if s["onto"] is not None else 0.0)


def _gemv_exact(s):
    c = s["c"]
    N, K, k = c["N"], c["K"], c["top_k"]
    x = s["x"].double()
    out = torch.zeros(s["d"].shape, dtype=torch.double, device=x.device)
    if s["base"] is not None:
        out += s["base"].double()
    magnitudes = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.double, device=x.device) / 2
    for e in range(c["groups"]):
        if k:
            at = (s["ids"].view(-1) == c["first"] + e).nonzero().view(-1)
            rows = at if c["per_choice"] else at // k
        else:
            at = rows = torch.arange(c["M"], device=x.device)
        if not at.numel():
            continue
        b = s["b"][e] if k else s["b"]
        w = torch.empty(N, K, dtype=torch.double, device=x.device)
        for half in (0, 1):
            q = (b.to(torch.int32) >> (4 * half)) & 15
            w[:, half::2] = magnitudes[q & 7] * (1 - 2 * (q >> 3)) if c["form"] == "fp4" else q.double()
        if c["form"] == "fp4":
            words = (s["sfb"][e] if k else s["sfb"]).long()
            for j in range(4):
                power = torch.ldexp(torch.ones(words.shape, dtype=torch.double, device=x.device),
                                    ((words >> (8 * j)) & 255) - 127)
                w.view(N, K // BLOCK, BLOCK)[:, :, 32 * j:32 * j + 32] *= power.t().unsqueeze(2)
        else:
            g = c["group"]
            w = w.view(N, K // g, g)
            zero = (s["zeros"][e] if k else s["zeros"]).double().t().unsqueeze(2) if s["zeros"] is not None else 8.0
            w = ((w - zero) * (s["scales"][e] if k else s["scales"]).double().t().unsqueeze(2)).view(N, K)
        out[at] += x[rows] @ w.t()
    return out


def _clip_exact(s):
    f, h = s["f"].double(), s["h"].double()
    norm = torch.sqrt(f.dot(f) + h.dot(h))
    factor = torch.clamp(s["max_norm"] / (norm + TINY_NORM), max=1.0)
    return {"norm": norm.view(1), "f": f * factor, "h": h * factor}


def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _balance_exact, "gemv": _gemv_exact, "clip": _clip_exact}[case["op"]](s)
