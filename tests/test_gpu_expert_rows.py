"""The rows' way out and back against the fp64 oracle: layouts exactly, scales
to the last bits, every code the nearest one, sums within bounds derived from
fp32 accumulation and one bf16 rounding."""
import numpy as np
import pytest
import torch

import oracle
from oracle import around
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

KEEP = 0xA5                      # code left where nothing may be written


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def choices(rng, T, k, experts, absent=0.05):
    ids = np.stack([rng.permutation(experts)[:k] for _ in range(T)]) if T else np.zeros((0, k), dtype=np.int64)
    ids = ids.astype(np.int32)
    ids[rng.random(ids.shape) < absent] = -1
    return ids


def i32(*shape, fill=-9):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def layout(dg, ids, first, G, M):
    T, k = ids.shape
    out = i32(M), i32(T, k), i32(M), i32(G)
    dg.dg_m_grouped_layout_contiguous(dev(ids), first, *out)
    torch.cuda.synchronize()
    return out


def masked_layout(dg, ids, first, G, max_m):
    T, k = ids.shape
    out = i32(G), i32(T, k), i32(G, max_m)
    dg.dg_m_grouped_layout_masked(dev(ids), first, *out)
    torch.cuda.synchronize()
    return out


SHAPES = [
    # T, top_k, experts, first, groups
    (0, 2, 4, 0, 4), (1, 1, 1, 0, 1), (1, 8, 256, 0, 256), (3, 2, 8, 0, 8), (64, 8, 128, 32, 32), (127, 3, 9, 2, 5),
    (129, 6, 64, 0, 64), (1000, 8, 31, 7, 17), (2049, 1, 3, 0, 3), (4096, 2, 8, 0, 8), (9001, 4, 257, 0, 257),
    (700, 4, 1024, 0, 1024), (40000, 6, 160, 16, 80),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layout_contiguous(dg, shape):
    T, k, experts, first, G = shape
    print(f"case: contiguous layout {shape}", flush=True)
    ids = choices(np.random.default_rng(T + k), T, k, experts)
    bound = dg.dg_m_grouped_rows_bound(T * k, G)
    assert bound == around.rows_bound(T * k, G)
    for M in {bound, max(0, bound // 256 * 128), 0, bound + 256}:
        got = layout(dg, ids, first, G, M)
        for g, r, what in zip(got, around.layout_contiguous(ids, first, G, M), ("layout", "row_of", "slot_of", "counts")):
            assert np.array_equal(g.cpu().numpy(), r), (what, M)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layout_masked(dg, shape):
    T, k, experts, first, G = shape
    print(f"case: masked layout {shape}", flush=True)
    ids = choices(np.random.default_rng(T + k + 1), T, k, experts)
    for max_m in {0, 1, T * k // G // 2 + 1, T + 3}:
        got = masked_layout(dg, ids, first, G, max_m)
        for g, r, what in zip(got, around.layout_masked(ids, first, G, max_m), ("masked_m", "row_of", "slot_of")):
            assert np.array_equal(g.cpu().numpy(), r), (what, max_m)


def test_layout_one_expert_takes_all_and_extreme_ids(dg):
    print("case: layouts of one expert and of ids beyond the experts", flush=True)
    ids = np.zeros((5000, 1), dtype=np.int32)
    for first, G in ((0, 1), (0, 3), (-2, 3)):
        got = layout(dg, ids, first, G, 5120)
        for g, r in zip(got, around.layout_contiguous(ids, first, G, 5120)):
            assert np.array_equal(g.cpu().numpy(), r)
    ids = np.array([[2**31 - 1, -2**31, 5], [4, 6, -1]], dtype=np.int32)
    for first in (5, -2**31, 2**31 - 1):
        got = layout(dg, ids, first, 2, 256)
        for g, r in zip(got, around.layout_contiguous(ids, first, 2, 256)):
            assert np.array_equal(g.cpu().numpy(), r)


@pytest.mark.parametrize("ws", [0, 4096, 1 << 16])
def test_layout_with_a_small_bound_workspace(dg, ws):
    print(f"case: layout on a stream with a workspace of {256 + ws} bytes", flush=True)
    ids = choices(np.random.default_rng(1), 9000, 4, 64)
    M = dg.dg_m_grouped_rows_bound(ids.size, 64)
    st = torch.cuda.Stream()
    buf = torch.zeros(256 + ws, dtype=torch.uint8, device="cuda")
    dg.dg_bind_stream_workspace(st, buf)
    try:
        out = i32(M), i32(9000, 4), i32(M), i32(64)
        d = dev(ids)
        torch.cuda.synchronize()
        dg.dg_m_grouped_layout_contiguous(d, 0, *out, stream=st)
        st.synchronize()
    finally:
        dg.dg_bind_stream_workspace(st, None)
    for g, r in zip(out, around.layout_contiguous(ids, 0, 64, M)):
        assert np.array_equal(g.cpu().numpy(), r)


def check_codes(codes, sf, v, amax, pow2, what):
    """codes and sf (broadcast to v) of the values v with block maxima amax, all fp64."""
    want = around.block_scales(amax, pow2)
    # one fp32 division; under pow2 the fp32 quotient picks the power
    assert np.all(np.abs(sf - want) <= (0.0 if pow2 else 2.0 ** -23) * want), what
    q = oracle.decode_e4m3(codes).astype(np.float64)
    u = v / sf
    # fp32: weight times value, 1 / sf and their product round to 2^-24 each
    near = 0.5 * around.e4m3_step(u) + 4 * 2.0 ** -24 * np.abs(u)
    assert np.all(np.abs(q - np.clip(u, -448.0, 448.0)) <= near), what


def rows_input(rng, T, K):
    """Rows with blocks of every kind: ordinary, all zero, one value, tiny, subnormal, large."""
    x = rng.standard_normal((T, K)).astype(np.float32)
    for t in range(T):
        for kb in range(K // 128):
            b = x[t, kb * 128:(kb + 1) * 128]
            kind = (t * 5 + kb) % 11
            if kind == 1:
                b[:] = 0.0
            elif kind == 3:
                b[1:] = 0.0
            elif kind == 5:
                b *= 2.0 ** -110
            elif kind == 6:
                b *= 2.0 ** -128
            elif kind == 7:
                b *= 2.0 ** 100
            elif kind == 9:
                b[:] = 448.0 * 2.0 ** rng.integers(-6, 6)
    return torch.from_numpy(x).to(torch.bfloat16)


SCATTER = [
    # T, top_k, experts, first, groups, K
    (1, 1, 1, 0, 1, 128), (1, 8, 16, 0, 16, 7168), (5, 2, 8, 0, 8, 384), (64, 8, 128, 32, 32, 512),
    (77, 3, 6, 1, 4, 1408), (300, 2, 8, 0, 8, 1152), (515, 6, 40, 0, 40, 256), (9, 4, 4, 0, 4, 16384),
    (2100, 1, 5, 0, 5, 128), (2050, 8, 24, 0, 24, 640),
]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("shape", SCATTER, ids=str)
def test_scatter(dg, shape, weighted, pow2):
    T, k, experts, first, G, K = shape
    print(f"case: scatter {shape} weighted={weighted} pow2={pow2}", flush=True)
    rng = np.random.default_rng(K + T)
    ids = choices(rng, T, k, experts)
    x = rows_input(rng, T, K)
    w = (rng.random((T, k)).astype(np.float32) - 0.3) if weighted else None
    xv = x.double().numpy()
    wd = None if w is None else dev(w)
    for form in ("contiguous", "masked"):
        if form == "contiguous":
            M = dg.dg_m_grouped_rows_bound(T * k, G)
            _, row_of, slot_of, _ = layout(dg, ids, first, G, M)
            a = torch.full((M, K), KEEP, dtype=torch.uint8, device="cuda")
            sfa = torch.full((K // 128, M), -3.0, device="cuda")
            dg.dg_m_grouped_scatter_fp8_contiguous(x.cuda(), wd, row_of, slot_of, a, sfa, pow2_scales=pow2)
            torch.cuda.synchronize()
            codes, sf = a.cpu().numpy(), sfa.cpu().numpy().T
        else:
            m = max(1, T * k // G)
            _, row_of, slot_of = masked_layout(dg, ids, first, G, m)
            a = torch.full((G, m, K), KEEP, dtype=torch.uint8, device="cuda")
            sfa = torch.full((G, K // 128, m), -3.0, device="cuda")
            dg.dg_m_grouped_scatter_fp8_masked(x.cuda(), wd, row_of, slot_of, a, sfa, pow2_scales=pow2)
            torch.cuda.synchronize()
            codes, sf = a.cpu().numpy().reshape(G * m, K), sfa.cpu().numpy().transpose(0, 2, 1).reshape(G * m, K // 128)
        slot = slot_of.cpu().numpy().ravel()
        free = slot < 0
        assert np.all(codes[free] == KEEP) and np.all(sf[free] == -3.0)
        rows = np.nonzero(~free)[0]
        v = xv[slot[rows] // k]
        if weighted:         # the fp32 product is the value that is quantised
            v = (x.float().numpy()[slot[rows] // k] * w.ravel()[slot[rows], None]).astype(np.float64)
        vb = v.reshape(rows.size, K // 128, 128)
        amax = np.abs(vb).max(axis=2)
        s = sf[rows].astype(np.float64)
        if pow2:             # the power is chosen from the fp32 quotient
            amax = (amax.astype(np.float32) / np.float32(448.0)).astype(np.float64) * 448.0
        check_codes(codes[rows].reshape(vb.shape), s[:, :, None], vb, amax[:, :, None], pow2, form)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16), (5, 2, 4, 48), (300, 2, 8, 256), (129, 3, 5, 1040), (64, 8, 32, 144)],
                         ids=str)
def test_kgrouped_scatter(dg, shape, weighted, pow2):
    T, k, G, N = shape
    print(f"case: K-grouped scatter {shape} weighted={weighted} pow2={pow2}", flush=True)
    rng = np.random.default_rng(N + T)
    ids = choices(rng, T, k, G)
    x = bf16(rng, T, N)
    x[:, ::5] *= 0.0
    w = (rng.random((T, k)).astype(np.float32) - 0.3) if weighted else None
    M = dg.dg_m_grouped_rows_bound(T * k, G)
    _, _, slot_of, _ = layout(dg, ids, 0, G, M)
    a = torch.full((M, N), KEEP, dtype=torch.uint8, device="cuda")
    sfa = torch.full((M // 128, N), -3.0, device="cuda")
    dg.dg_k_grouped_scatter_fp8(x.cuda(), None if w is None else dev(w), slot_of, k, a, sfa, pow2_scales=pow2)
    torch.cuda.synchronize()
    slot = slot_of.cpu().numpy()
    v = x.float().numpy()[np.maximum(slot, 0) // k]
    if weighted:
        v = v * w.ravel()[np.maximum(slot, 0), None]
    v = np.where(slot[:, None] >= 0, v, np.float32(0)).astype(np.float64).reshape(M // 128, 128, N)
    amax = np.abs(v).max(axis=1)
    if pow2:
        amax = (amax.astype(np.float32) / np.float32(448.0)).astype(np.float64) * 448.0
    sf = sfa.cpu().numpy().astype(np.float64)
    check_codes(a.cpu().numpy().reshape(v.shape), sf[:, None, :], v, amax[:, None, :], pow2, "k-grouped")
    assert np.all(a.cpu().numpy()[slot < 0] == 0)


def test_scatter_of_nonfinite_values(dg):
    print("case: scatter of NaN and infinities", flush=True)
    x = torch.ones(4, 256, dtype=torch.bfloat16)
    x[0, 3], x[1, 5], x[2, 130] = float("nan"), float("inf"), float("-inf")
    x[3, :128] = float("nan")
    ids = np.zeros((4, 1), dtype=np.int32)
    _, row_of, slot_of, _ = layout(dg, ids, 0, 1, 128)
    a = torch.zeros(128, 256, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(2, 128, device="cuda")
    dg.dg_m_grouped_scatter_fp8_contiguous(x.cuda(), None, row_of, slot_of, a, sfa)
    torch.cuda.synchronize()
    c, s = a.cpu().numpy()[:4], sfa.cpu().numpy()[:, :4]
    nan = (c & 0x7F) == 0x7F
    assert nan.sum() == 3 + 128 and nan[0, 3] and nan[1, 5] and nan[2, 130] and nan[3, :128].all()
    assert s[0, 0] == np.float32(1.0) / np.float32(448.0) and np.isinf(s[0, 1]) and np.isinf(s[1, 2])
    assert s[0, 3] == 1.0
    assert np.all(c[0, [0, 1, 200]] == 0x7E)        # 448 at scale amax / 448


def test_scatter_skips_entries_out_of_range(dg):
    print("case: scatter with map entries out of range", flush=True)
    x = torch.ones(3, 128, dtype=torch.bfloat16, device="cuda")
    row_of = torch.tensor([[1, 500], [-5, 2**31 - 1], [3, -1]], dtype=torch.int32, device="cuda")
    slot_of = torch.tensor([-2**31, 0, 6, 4], dtype=torch.int32, device="cuda")
    a = torch.full((4, 128), KEEP, dtype=torch.uint8, device="cuda")
    sfa = torch.full((1, 4), -3.0, device="cuda")
    dg.dg_m_grouped_scatter_fp8_contiguous(x, None, row_of, slot_of, a, sfa)
    torch.cuda.synchronize()
    got = a.cpu().numpy()
    assert np.all(got[[0, 2]] == KEEP) and np.all(got[[1, 3]] == 0x7E)
    assert np.all(sfa.cpu().numpy()[0, [0, 2]] == -3.0)


GATHER = [
    # T, top_k, M, N
    (1, 1, 1, 1), (1, 8, 128, 7168), (3, 2, 256, 24), (64, 8, 640, 513), (65, 4, 300, 2047), (5, 64, 90, 130),
    (33, 3, 128, 1000), (257, 1, 128, 129), (2, 2, 4, 16385), (40, 6, 512, 2112),
]


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("residual", ["none", "c", "in place"])
@pytest.mark.parametrize("shape", GATHER, ids=str)
def test_gather(dg, shape, weighted, residual):
    T, k, M, N = shape
    print(f"case: gather {shape} weighted={weighted} residual={residual}", flush=True)
    rng = np.random.default_rng(N + T)
    rows = bf16(rng, M, N)
    at = rng.integers(0, M, (T, k)).astype(np.int32)
    at[rng.random((T, k)) < 0.2] = -1
    at[0, -1] = M                                   # just beyond the rows
    if T > 1:
        at[1] = -1                                  # a token without any row
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    if weighted:
        w[(at < 0) | (at >= M)] = np.nan            # what weighs nothing is not read
    c = None if residual == "none" else bf16(rng, T, N)
    d = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    if residual == "in place":
        d.copy_(c)
    cd = None if c is None else d if residual == "in place" else c.cuda()
    dg.dg_m_grouped_gather(rows.cuda(), dev(at), None if w is None else dev(w), cd, d)
    torch.cuda.synchronize()
    ref, mag = around.gather(rows.float().numpy(), at, w, None if c is None else c.float().numpy())
    err = np.abs(d.float().cpu().numpy() - ref)
    # k + 1 fp32 roundings of partial sums, then one to bf16
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + (k + 1) * 2.0 ** -23 * mag + 1e-37)


def test_gather_takes_the_masked_form(dg):
    print("case: gather from [G][max_m][N]", flush=True)
    rng = np.random.default_rng(2)
    rows = bf16(rng, 4, 9, 40)
    at = rng.integers(-1, 36, (21, 3)).astype(np.int32)
    d = torch.empty(21, 40, dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_gather(rows.cuda(), dev(at), None, None, d)
    torch.cuda.synchronize()
    ref, mag = around.gather(rows.float().numpy().reshape(36, 40), at, None, None)
    assert np.all(np.abs(d.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * mag)


def test_gather_does_not_read_rows_it_does_not_sum(dg):
    print("case: gather beside NaN rows", flush=True)
    rows = torch.full((6, 264), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[2] = 1.5
    at = torch.tensor([[2, -1, 6], [-1, -1, -1], [-2, 2, 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 0.0, 0.0], [1.0, 1.0, 1.0], [float("inf"), 2.0, 3.0]], device="cuda")
    d = torch.empty(3, 264, dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_gather(rows, at, w, None, d)
    gw = torch.full((3, 3), -1.0, device="cuda")
    dg.dg_m_grouped_gather_weight_grad(rows, at, torch.ones_like(d), gw)
    torch.cuda.synchronize()
    assert torch.equal(d.float().cpu(), torch.tensor([1.5, 0.0, 7.5]).unsqueeze(1).expand(3, 264))
    assert torch.equal(gw.cpu(), torch.tensor([[396.0, 0, 0], [0, 0, 0], [0, 396.0, 396.0]]))


@pytest.mark.parametrize("shape", GATHER, ids=str)
def test_gather_weight_gradient(dg, shape):
    T, k, M, N = shape
    print(f"case: gather weight gradient {shape}", flush=True)
    rng = np.random.default_rng(N * 3 + T)
    rows, g = bf16(rng, M, N), bf16(rng, T, N)
    at = rng.integers(0, M, (T, k)).astype(np.int32)
    at[rng.random((T, k)) < 0.2] = -1
    at[0, -1] = M
    out = torch.full((T, k), float("nan"), device="cuda")
    dg.dg_m_grouped_gather_weight_grad(rows.cuda(), dev(at), g.cuda(), out)
    torch.cuda.synchronize()
    ref, mag = around.gather_weight_grad(rows.float().numpy(), at, g.float().numpy())
    # products of bf16 are exact in fp32; N additions in any order
    assert np.all(np.abs(out.cpu().numpy() - ref) <= N * 2.0 ** -24 * mag + 1e-37)


def test_weight_gradient_against_differences(dg):
    print("case: gather weight gradient by differences", flush=True)
    rng = np.random.default_rng(8)
    rows, g = bf16(rng, 20, 72), bf16(rng, 6, 72)
    at = rng.integers(-1, 20, (6, 3)).astype(np.int32)
    out = torch.empty(6, 3, device="cuda")
    dg.dg_m_grouped_gather_weight_grad(rows.cuda(), dev(at), g.cuda(), out)
    torch.cuda.synchronize()
    r, gd = rows.float().numpy(), g.double().numpy()
    w = rng.standard_normal((6, 3))
    for j in range(3):
        dw = np.zeros((6, 3))
        dw[:, j] = 1.0                              # the gather is linear in its weights
        up, down = around.gather(r, at, w + dw, None)[0], around.gather(r, at, w - dw, None)[0]
        ref = ((up - down) / 2 * gd).sum(axis=1)
        assert np.all(np.abs(out[:, j].cpu().numpy() - ref) <= 72 * 2.0 ** -22)


def test_gather_and_scatter_are_adjoint(dg):
    # <gather(rows), y> = <rows, scatter(y)> up to the scatter's e4m3 rounding:
    # half a step of 2^-3 relative, 2^-4 of the block's values at most
    print("case: the scatter is the gather's adjoint", flush=True)
    rng = np.random.default_rng(4)
    T, k, G, K = 50, 3, 7, 256
    ids = choices(rng, T, k, G, absent=0.1)
    M = dg.dg_m_grouped_rows_bound(T * k, G)
    _, row_of, slot_of, _ = layout(dg, ids, 0, G, M)
    y, rows = bf16(rng, T, K), bf16(rng, M, K)
    w = rng.random((T, k)).astype(np.float32) + 0.1
    a = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    sfa = torch.ones(K // 128, M, device="cuda")
    dg.dg_m_grouped_scatter_fp8_contiguous(y.cuda(), dev(w), row_of, slot_of, a, sfa)
    torch.cuda.synchronize()
    s = oracle.decode_e4m3(a.cpu().numpy()).reshape(M, K // 128, 128) * sfa.cpu().numpy().T[:, :, None]
    s = s.reshape(M, K)
    at = row_of.cpu().numpy()
    d, _ = around.gather(rows.float().numpy(), at, w, None)
    left, right = (d * y.double().numpy()).sum(), (rows.double().numpy() * s).sum()
    size = (np.abs(rows.double().numpy()) * np.abs(s)).sum()
    assert abs(left - right) <= 2.0 ** -4 * size
    assert abs(left - right) <= 5 * 2.0 ** -4 * np.sqrt((rows.double().numpy() ** 2 * s ** 2).sum())


def test_gather_of_more_tokens_than_a_grid_axis(dg):
    print("case: gather of 70001 tokens", flush=True)
    rng = np.random.default_rng(6)
    T, k, M, N = 70001, 2, 500, 9
    rows = bf16(rng, M, N)
    at = rng.integers(-1, M + 1, (T, k)).astype(np.int32)
    d = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_gather(rows.cuda(), dev(at), None, None, d)
    gw = torch.full((T, k), float("nan"), device="cuda")
    dg.dg_m_grouped_gather_weight_grad(rows.cuda(), dev(at), d, gw)
    torch.cuda.synchronize()
    ref, mag = around.gather(rows.float().numpy(), at, None, None)
    assert np.all(np.abs(d.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 1) * 2.0 ** -23 * mag + 1e-37)
    ref, mag = around.gather_weight_grad(rows.float().numpy(), at, d.float().cpu().numpy())
    assert np.all(np.abs(gw.cpu().numpy() - ref) <= N * 2.0 ** -24 * mag + 1e-37)


@pytest.mark.parametrize("weighted", [False, True])
def test_scatter_of_many_rows_without_room_for_the_maxima(dg, weighted):
    # from 32768 rows on the scales are written row by row from maxima in the
    # workspace; with a bound one too small for them, as for fewer rows: the same bits
    print(f"case: scatter of 40064 rows with a small bound workspace, weighted={weighted}", flush=True)
    rng = np.random.default_rng(7)
    T, k, G, K = 10000, 4, 3, 384
    ids = np.stack([rng.permutation(4)[:k] for _ in range(T)]).astype(np.int32)
    x = bf16(rng, T, K).cuda()
    w = dev(rng.standard_normal((T, k)).astype(np.float32)) if weighted else None
    M = 40064
    _, row_of, slot_of, _ = layout(dg, ids, 0, G, M)
    outs = []
    st = torch.cuda.Stream()
    buf = torch.empty(512, dtype=torch.uint8, device="cuda")
    for stream in (None, st):
        a = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
        sfa = torch.zeros(K // 128, M, device="cuda")
        torch.cuda.synchronize()
        if stream is not None:
            dg.dg_bind_stream_workspace(stream, buf)
        try:
            dg.dg_m_grouped_scatter_fp8_contiguous(x, w, row_of, slot_of, a, sfa, stream=stream)
            torch.cuda.synchronize()
        finally:
            if stream is not None:
                dg.dg_bind_stream_workspace(stream, None)
        outs.append((a, sfa))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert int((outs[0][1] != 0).sum()) == int((slot_of >= 0).sum()) * (K // 128)
