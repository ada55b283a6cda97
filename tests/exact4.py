"""Products with 4-bit weights whose sums are exact in fp32 in any order: x is whole
numbers of -2 to 2, c multiples of a quarter, FP4 exponents 2^-1 to 2^1 and integers'
scales 1/2 to 2.  All terms of E2M1 are multiples of 1/4 of at most 24 in magnitude,
those of integers (q - zero, and q and zero apart) multiples of 1/2 of at most 60: with
K up to 16512 all sums of any of them, with c, stay below 2^22 of these units, and fp32
holds 2^24.  A result is then the one nearest bf16 value, to the bit: a value of K that
is left out, taken twice or scaled by its neighbour's scale shows."""
import torch

from oracle import layer

FORMS = ["fp4", ("int4", 32, "float32", True), ("int4", 32, "bfloat16", False), ("int4", 64, "bfloat16", True),
         ("int4", 64, "float32", False), ("int4", 128, "float32", True), ("int4", 128, "bfloat16", False)]


def generator(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def draw(g, low, high, *shape, dtype=torch.uint8):
    return torch.randint(low, high, shape, device=g.device, generator=g, dtype=dtype)


def whole(g, *shape):
    return draw(g, -2, 3, *shape, dtype=torch.int8).to(torch.bfloat16)


def quarters(g, *shape):
    return (draw(g, -128, 129, *shape, dtype=torch.int32) / 4).to(torch.bfloat16)


def weights(g, form, lead, N, K):
    """The products' arguments after x."""
    b = draw(g, 0, 256, *lead, N, K // 2)
    if form == "fp4":
        return b, draw(g, 126, 129, *lead, K // 128, N, 4).view(torch.int32).squeeze(-1)
    _, group, dtype, with_zeros = form
    s = torch.exp2(draw(g, -1, 2, *lead, K // group, N, dtype=torch.int8).float())
    return b, s.to(getattr(torch, dtype)), draw(g, 0, 16, *s.shape) if with_zeros else None


def of_expert(args, e):
    return [None if t is None else t[e] for t in args]


LEVELS = torch.tensor(layer.E2M1)


def decode(form, b, scale, zeros=None):
    """The weights [N][K] in fp64, on the tensors' device."""
    N, K = b.shape[0], 2 * b.shape[1]
    q = torch.stack([b & 15, b >> 4], -1).view(N, K)
    if form == "fp4":
        e = scale.view(torch.uint8).view(K // 128, N, 4).permute(1, 0, 2).reshape(N, K // 32, 1)
        w = LEVELS.to(b.device)[q.long()].view(N, K // 32, 32)
        return (w * torch.exp2(e.double() - 127.0)).view(N, K)
    group = form[1]
    z = 8.0 if zeros is None else zeros.t().double().unsqueeze(2)
    return ((q.view(N, K // group, group).double() - z) * scale.t().double().unsqueeze(2)).view(N, K)


def product(x, w, c=None):
    """The nearest bf16 values of c + x w^T."""
    d = x.double() @ w.t()
    return (d if c is None else d + c.double()).to(torch.bfloat16)
