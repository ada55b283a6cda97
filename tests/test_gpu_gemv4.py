"""Products of a few tokens with 4-bit weights against the fp64 oracle: every term
is exact, sums over K are fp32 in any order (at most K + K / 16 + 16 of them, each
off by 2^-23 of the terms' magnitudes at most), one rounding to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

from oracle import layer
from tests.gpu_util import dev, sentinel_like

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def weights(rng, form, lead, N, K):
    """form: "fp4", or ("int4", group, scales' type, zeros); (the binding's arguments, [lead][N][K] in fp64, magnitudes)"""
    b = rng.integers(0, 256, (*lead, N, K // 2), dtype=np.uint8)
    count = int(np.prod(lead))
    flat = b.reshape(count, N, K // 2)
    if form == "fp4":
        e = rng.integers(115, 125, (count, K // 128, N, 4), dtype=np.uint8)
        sfb = e.view(np.int32).reshape(count, K // 128, N)
        w = [layer.fp4_weights(flat[g], sfb[g]) for g in range(count)]
        return (dev(b), dev(sfb.reshape(*lead, K // 128, N))), w, [np.abs(v) for v in w]
    _, group, dtype, with_zeros = form
    s = torch.from_numpy((0.01 * (rng.random((count, K // group, N)) + 0.5)).astype(np.float32)).to(getattr(torch, dtype))
    z = rng.integers(0, 16, (count, K // group, N), dtype=np.uint8) if with_zeros else None
    both = [layer.int4_weights(flat[g], s[g].double().numpy(), None if z is None else z[g]) for g in range(count)]
    args = (dev(b), s.reshape(*lead, K // group, N).cuda(), None if z is None else dev(z.reshape(*lead, K // group, N)))
    return args, [v[0] for v in both], [v[1] for v in both]


def check(got, ref, mag, K, what=""):
    assert np.all(np.isfinite(got)), what
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * np.abs(ref) + (K + K // 16 + 16) * 2.0 ** -23 * mag + 1e-37
    assert np.all(err <= bound), (what, float((err / bound).max()))


FORMS = ["fp4", ("int4", 32, "float32", True), ("int4", 64, "bfloat16", False), ("int4", 128, "bfloat16", True),
         ("int4", 128, "float32", False)]
SIZES = [
    # M, N, K
    (1, 1, 128), (1, 16, 128), (1, 2112, 7168), (2, 17, 256), (3, 100, 384), (5, 129, 640), (8, 513, 1024),
    (15, 64, 1408), (16, 1000, 896), (17, 31, 2048), (33, 2047, 256), (64, 96, 4224), (1, 24, 16384), (100, 7, 128),
    (7, 4097, 128), (9, 300, 7168), (31, 48, 1152), (4, 2112, 512),
]


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_dense(dg, size, form):
    M, N, K = size
    print(f"case: gemv {size} {form}", flush=True)
    rng = np.random.default_rng(M + N + K)
    args, w, mag_w = weights(rng, form, (), N, K)
    call = dg.dg_bf16_fp4_gemv_nt if form == "fp4" else dg.dg_bf16_int4_gemv_nt
    x, c = bf16(rng, M, K), bf16(rng, M, N)
    for with_c in (False, True):
        d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        call(x.cuda(), *args, c.cuda() if with_c else None, d)
        torch.cuda.synchronize()
        ref, mag = layer.gemv(x.double().numpy(), w[0], c.double().numpy() if with_c else None, mag_w[0])
        check(d.double().cpu().numpy(), ref, mag, K, (size, form, with_c))


CHOICES = [
    # T, top_k, experts in all, first here, here, N, K, a row of x per choice
    (1, 1, 1, 0, 1, 1, 128, False), (1, 8, 16, 0, 16, 100, 256, True), (1, 8, 32, 8, 8, 2112, 512, False),
    (5, 3, 9, 3, 3, 129, 384, False), (64, 8, 128, 32, 32, 40, 256, False), (64, 8, 8, 0, 8, 33, 128, True),
    (40, 1, 2, 0, 1, 65, 640, False), (65, 8, 16, 4, 8, 24, 128, False), (300, 4, 5, 0, 5, 50, 256, True),
    (2000, 2, 40, 0, 40, 17, 128, False), (513, 1, 1, 0, 1, 31, 128, False), (7, 2, 64, 60, 4, 513, 1024, True),
    (128, 4, 1024, 0, 1024, 8, 128, False),
]


def choices(rng, T, k, experts):
    ids = np.argsort(rng.random((T, experts)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < 0.05] = -1
    return ids


@pytest.mark.parametrize("form", FORMS[:3], ids=str)
@pytest.mark.parametrize("case", CHOICES, ids=lambda s: "-".join(map(str, s)))
def test_by_choice(dg, case, form):
    T, k, experts, first, G, N, K, per_choice = case
    print(f"case: gemv by choice {case} {form}", flush=True)
    rng = np.random.default_rng(T + k + N + K)
    args, w, mag_w = weights(rng, form, (G,), N, K)
    call = dg.dg_m_grouped_bf16_fp4_gemv_nt_topk if form == "fp4" else dg.dg_m_grouped_bf16_int4_gemv_nt_topk
    ids = choices(rng, T, k, experts)
    x, c = bf16(rng, T * k if per_choice else T, K), bf16(rng, T * k, N)
    for with_c in (False, True):
        d = torch.full((T * k, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        if with_c:
            d.copy_(c)
        call(x.cuda(), dev(ids), first, *args, d if with_c else None, d)
        torch.cuda.synchronize()
        got = d.double().cpu().numpy()
        xs = x.double().numpy()[np.arange(T * k) if per_choice else np.repeat(np.arange(T), k)]
        cs = c.double().numpy()
        flat = ids.ravel() - first
        for e in range(-1, G):
            at = np.nonzero(flat == e if e >= 0 else (flat < 0) | (flat >= G))[0]
            if e < 0:
                assert np.array_equal(got[at], cs[at] if with_c else np.zeros((len(at), N)))
            elif len(at):
                ref, mag = layer.gemv(xs[at], w[e], cs[at] if with_c else None, mag_w[e])
                check(got[at], ref, mag, K, (case, form, with_c, e))


def test_column_slices_and_neighbours(dg):
    """x, c and d as column slices of wider arrays at odd column numbers; what lies around d stays."""
    rng = np.random.default_rng(7)
    for M, N, K in ((3, 37, 256), (20, 130, 384)):
        args, w, mag_w = weights(rng, "fp4", (), N, K)
        x, c = bf16(rng, M, K + 24), bf16(rng, M, N + 5)
        wide = sentinel_like((M + 2, N + 9))
        before = wide.clone()
        dg.dg_bf16_fp4_gemv_nt(x.cuda()[:, 8:8 + K], *args, c.cuda()[:, 3:3 + N], wide[1:M + 1, 5:5 + N])
        torch.cuda.synchronize()
        ref, mag = layer.gemv(x[:, 8:8 + K].double().numpy(), w[0], c[:, 3:3 + N].double().numpy(), mag_w[0])
        check(wide[1:M + 1, 5:5 + N].double().cpu().numpy(), ref, mag, K)
        wide[1:M + 1, 5:5 + N] = before[1:M + 1, 5:5 + N]
        assert torch.equal(wide.view(torch.int16), before.view(torch.int16))


def test_in_place(dg):
    rng = np.random.default_rng(8)
    args, w, mag_w = weights(rng, ("int4", 64, "float32", True), (), 77, 512)
    x, c = bf16(rng, 19, 512), bf16(rng, 19, 77)
    d = c.cuda()
    dg.dg_bf16_int4_gemv_nt(x.cuda(), *args, d, d)
    ref, mag = layer.gemv(x.double().numpy(), w[0], c.double().numpy(), mag_w[0])
    check(d.double().cpu().numpy(), ref, mag, 512)


def test_every_code_and_every_exponent(dg):
    """One-hot x picks single weights: all 16 codes, exponents to both ends of bf16."""
    K, N = 128, 16
    codes = np.tile(np.arange(16, dtype=np.uint8)[:, None], (1, K))
    b = (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
    x = torch.zeros(1, K, dtype=torch.bfloat16)
    x[0, 37] = 1.0
    for e in list(range(0, 10)) + [60, 126, 127, 128, 200, 250, 251, 252, 253, 254, 255]:
        sfb = np.full((1, N), e * 0x01010101, dtype=np.uint32).view(np.int32)
        d = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
        dg.dg_bf16_fp4_gemv_nt(x.cuda(), dev(b), dev(sfb), None, d)
        got = d.cpu()
        if e == 255:
            assert torch.isnan(got).all()
            continue
        exact = layer.E2M1 * 2.0 ** (e - 127)
        want = torch.from_numpy(exact).to(torch.bfloat16)        # subnormal down to 2^-133
        zero, far = (exact == 0), ~torch.isfinite(want).numpy()
        assert torch.equal(got[0][~zero & ~far], want[~zero & ~far]) and (got[0][zero] == 0).all(), (e, got, want)
        assert torch.isnan(got[0][far]).all()                    # infinite weights, also at the zeros of x
    # integers, every q and zero point
    q = np.tile(np.arange(16, dtype=np.uint8)[:, None], (1, K))
    b = (q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8)
    for z in range(16):
        for k in (0, 1, 2, 3, 4, 5, 6, 7, 31, 32, 63, 95, 127):
            x = torch.zeros(1, K, dtype=torch.bfloat16)
            x[0, k] = 1.0
            d = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
            dg.dg_bf16_int4_gemv_nt(x.cuda(), dev(b), dev(np.full((4, N), 0.5, np.float32)),
                                    dev(np.full((4, N), z, np.uint8)), None, d)
            assert torch.equal(d.cpu()[0].double(), torch.arange(16).double() * 0.5 - 0.5 * z), (z, k)


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_every_place_of_k(dg, form):
    """x is one-hot at every k in turn, token by token: each weight comes from its own place with its own scale."""
    rng = np.random.default_rng(3)
    N, K = 21, 384
    args, w, _ = weights(rng, form, (), N, K)
    x = torch.eye(K, dtype=torch.bfloat16)
    d = torch.empty(K, N, dtype=torch.bfloat16, device="cuda")
    call = dg.dg_bf16_fp4_gemv_nt if form == "fp4" else dg.dg_bf16_int4_gemv_nt
    call(x.cuda(), *args, None, d)
    ref = w[0].T
    assert np.all(np.abs(d.double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref).clip(1e-30))


def test_a_token_of_infinities_stays_alone(dg):
    rng = np.random.default_rng(4)
    for form in (FORMS[0], FORMS[1]):
        args, w, mag_w = weights(rng, form, (), 40, 256)
        x = bf16(rng, 6, 256)
        bad = x.clone()
        bad[2] = float("inf")
        bad[4, 9] = float("nan")
        call = dg.dg_bf16_fp4_gemv_nt if form == "fp4" else dg.dg_bf16_int4_gemv_nt
        outs = []
        for v in (x, bad):
            d = torch.empty(6, 40, dtype=torch.bfloat16, device="cuda")
            call(v.cuda(), *args, None, d)
            outs.append(d.cpu())
        for t in (0, 1, 3, 5):
            assert torch.equal(outs[0][t], outs[1][t])
        assert torch.isnan(outs[1][4]).all() and not torch.isfinite(outs[1][2]).any()


def test_no_experts_here_and_no_terms(dg):
    ids = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    x = torch.ones(2, 128, dtype=torch.bfloat16, device="cuda")
    c = torch.randn(4, 9, device="cuda").to(torch.bfloat16)
    d = torch.empty_like(c)
    b, sfb = torch.zeros(0, 9, 64, dtype=torch.uint8, device="cuda"), torch.zeros(0, 1, 9, dtype=torch.int32, device="cuda")
    dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x, ids, 0, b, sfb, c, d)
    assert torch.equal(c, d)
    dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x, ids, 0, b, sfb, None, d)
    assert (d == 0).all()
    d = torch.empty(2, 9, dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_fp4_gemv_nt(x[:, :0], b.view(9, 0), sfb.view(0, 9), c[:2], d)
    assert torch.equal(c[:2], d)


def test_small_workspace(dg):
    """Without room for lists the choices go out 512 at a time: the same results."""
    rng = np.random.default_rng(5)
    args, _, _ = weights(rng, "fp4", (6,), 40, 256)
    ids = dev(choices(rng, 900, 3, 8))
    x = bf16(rng, 900, 256).cuda()
    want, got = (torch.empty(2700, 40, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x, ids, 1, *args, None, want)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    dg.dg_bind_stream_workspace(stream, ws)
    try:
        with torch.cuda.stream(stream):
            dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x, ids, 1, *args, None, got)
        torch.cuda.synchronize()
    finally:
        dg.dg_bind_stream_workspace(stream, None)
    assert torch.equal(got, want)
