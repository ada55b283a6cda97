"""The router's balance loss, its counts and its gradient against the fp64 oracle.

Bounds: an exponential is off by at most 2e-7 of itself, below 4 units of 2^-24; a
share has one of those, the sum over E of them, a reciprocal and a product, so at
most (E + 16) units; sums over tokens add at most 128 more at these sizes; every
term of the loss is positive, so its error is at most (E + 160) * 2^-24 of it.  The
gradient's two terms are measured by their magnitudes in the same way, and its
result is rounded once more to its type."""
import numpy as np
import pytest
import torch

from oracle import layer
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def problem(seed, T, E, k, S, dtype, masked=0.0, spread=1.5):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((T, E)) * spread).astype(np.float32)).to(getattr(torch, dtype))
    x[torch.from_numpy(rng.random((T, E)) < masked)] = -float("inf")
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32) if T else np.zeros((0, k), np.int32)
    ids[rng.random(ids.shape) < 0.05] = -1
    ids[rng.random(ids.shape) < 0.02] = E
    starts = None
    if S:
        starts = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    return rng, x, ids, starts


def forward(dg, x, ids, starts, score, scale=1.0):
    S = 1 if starts is None else len(starts) - 1
    E = x.shape[1]
    loss = torch.full((S,), float("nan"), device="cuda")
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    dg.dg_route_balance(x.cuda(), dev(ids), None if starts is None else dev(starts), loss, counts, score=score,
                        scale=scale)
    torch.cuda.synchronize()
    return loss.cpu().numpy().astype(np.float64), counts.cpu().numpy()


CASES = [
    # T, E, top_k, sequences (0: no seq_starts), type
    (1, 1, 1, 0, "float32"), (1, 8, 2, 1, "bfloat16"), (5, 7, 3, 3, "float32"), (16, 60, 4, 0, "bfloat16"),
    (17, 64, 6, 5, "float32"), (63, 65, 1, 2, "bfloat16"), (130, 128, 8, 40, "float32"), (257, 130, 10, 7, "bfloat16"),
    (300, 255, 8, 0, "float32"), (1000, 256, 8, 3, "float32"), (511, 257, 2, 90, "bfloat16"),
    (200, 512, 64, 4, "float32"), (129, 513, 8, 6, "bfloat16"), (70, 1024, 8, 2, "float32"), (3, 1023, 16, 5, "float32"),
    (9000, 16, 2, 2, "bfloat16"), (0, 16, 2, 3, "float32"), (40, 12, 12, 300, "float32"),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_loss_and_counts(dg, case, score):
    T, E, k, S, dtype = case
    print(f"case: balance {case} {score}", flush=True)
    _, x, ids, starts = problem(T + E, T, E, k, S, dtype, masked=0.05 if E > 8 else 0.0)
    loss, counts = forward(dg, x, ids, starts, score, scale=0.25)
    want, n = layer.balance(x.float().numpy(), ids, starts, score, scale=0.25)
    assert np.array_equal(counts, n)
    assert np.all(np.abs(loss - want) <= (E + 160) * UNIT * want), np.abs(loss - want).max()


@pytest.mark.parametrize("onto", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_gradient(dg, case, score, onto):
    T, E, k, S, dtype = case
    print(f"case: balance gradient {case} {score} onto={onto}", flush=True)
    rng, x, ids, starts = problem(T + E + 1, T, E, k, S, dtype, masked=0.05 if E > 8 else 0.0)
    _, counts = layer.balance(x.float().numpy(), ids, starts, score)
    counts = counts.astype(np.int32)
    grad_loss = rng.standard_normal(max(S, 1)).astype(np.float32) if T % 2 else None
    c = torch.from_numpy((rng.standard_normal((T, E)) * 0.1).astype(np.float32)).to(x.dtype) if onto else None
    out = torch.full((T, E), float("nan"), dtype=x.dtype, device="cuda")
    if onto:
        out.copy_(c)
    dg.dg_route_balance_backward(x.cuda(), dev(counts), None if starts is None else dev(starts),
                                 None if grad_loss is None else dev(grad_loss), out if onto else None, out, k,
                                 score=score, scale=3.0)
    torch.cuda.synchronize()
    want, mag = layer.balance_backward(x.float().numpy(), counts, starts, grad_loss,
                                       None if c is None else c.double().numpy(), k, score, scale=3.0)
    got = out.double().cpu().numpy()
    bound = HALF[dtype] * np.abs(want) + (E + 32) * UNIT * mag + UNIT * mag + 1e-37
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())


def test_gradient_against_differences(dg):
    T, E, k = 6, 10, 3
    _, x, ids, _ = problem(5, T, E, k, 0, "float32")
    starts = np.array([0, 2, 2, 5], dtype=np.int32)
    counts = layer.balance(x.numpy(), ids, starts, "sigmoid")[1].astype(np.int32)
    for score in ("softmax", "sigmoid"):
        out = torch.empty(T, E, device="cuda")
        dg.dg_route_balance_backward(x.cuda(), dev(counts), dev(starts), None, None, out, k, score=score)
        h = 1e-4
        for t in range(T):
            for e in range(E):
                lo, hi = x.double().numpy().copy(), x.double().numpy().copy()
                lo[t, e] -= h
                hi[t, e] += h

                def total(v):
                    p, _ = layer.shares(v, score)
                    return sum(E / (k * float(b - a) ** 2) * float(counts[s] @ p[a:b].sum(0))
                               for s, (a, b) in enumerate([(0, 2), (2, 2), (2, 5)]) if b > a)
                slope = (total(hi) - total(lo)) / (2 * h)
                assert abs(slope - float(out[t, e])) < 1e-5, (score, t, e)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(dg, score):
    """Rows of infinities and NaN, of far negative logits, of one logit that takes all; shares that are nearly 1."""
    E, k = 20, 4
    x = np.zeros((9, E), dtype=np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 3] = np.inf
    x[3] = -200.0 + np.arange(E)                 # sigmoids below the smallest fp32 number
    x[4] = -np.inf
    x[4, 7] = -300.0
    x[5, 2] = 17.0                               # takes nearly all of a softmax
    x[6] = np.finfo(np.float32).min
    x[7] = np.finfo(np.float32).max
    x[8, 5] = 60.0
    rng = np.random.default_rng(1)
    ids = np.argsort(rng.random((9, E)), axis=1)[:, :k].astype(np.int32)
    loss, counts = forward(dg, torch.from_numpy(x), ids, None, score)
    want, n = layer.balance(x, ids, None, score)
    assert np.array_equal(counts, n)
    assert np.all(np.abs(loss - want) <= (E + 160) * UNIT * want)
    out = torch.empty(9, E, device="cuda")
    dg.dg_route_balance_backward(torch.from_numpy(x).cuda(), dev(n.astype(np.int32)), None, None, None, out, k,
                                 score=score)
    want, mag = layer.balance_backward(x, n, None, None, None, k, score)
    got = out.double().cpu().numpy()
    bound = UNIT * np.abs(want) + (E + 33) * UNIT * mag + 1e-37
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())
    assert np.all(got[:2] == 0)


def test_a_share_of_nearly_one_keeps_its_gradient(dg):
    """The dominant expert's gradient is what the others leave: no difference of large numbers."""
    E = 8
    for gap in (10.0, 17.0, 30.0, 60.0):
        x = np.zeros((1, E), dtype=np.float32)
        x[0, 2] = gap
        counts = np.arange(E, dtype=np.int32).reshape(1, E) * 1000003
        out = torch.empty(1, E, device="cuda")
        dg.dg_route_balance_backward(torch.from_numpy(x).cuda(), dev(counts), None, None, None, out, 2)
        want, _ = layer.balance_backward(x, counts, None, None, None, 2, "softmax")
        got = out.double().cpu().numpy()
        assert abs(got[0, 2] - want[0, 2]) <= 64 * UNIT * abs(want[0, 2]), gap


def test_padding_is_left_out(dg):
    T, E, k = 50, 24, 4
    _, x, ids, _ = problem(3, T, E, k, 0, "float32")
    starts = np.array([7, 20, 41], dtype=np.int32)
    loss, counts = forward(dg, x, ids, starts, "softmax")
    x2, ids2 = x.clone(), ids.copy()
    x2[:7], x2[41:] = float("nan"), float("inf")
    ids2[:7], ids2[41:] = 0, 1
    loss2, counts2 = forward(dg, x2, ids2, starts, "softmax")
    assert np.array_equal(loss, loss2) and np.array_equal(counts, counts2)
    c = torch.randn(T, E)
    out = torch.empty(T, E, device="cuda")
    dg.dg_route_balance_backward(x2.cuda(), dev(counts), dev(starts), None, c.cuda(), out, k)
    got = out.cpu()
    assert torch.equal(got[:7], c[:7]) and torch.equal(got[41:], c[41:])
    assert not torch.equal(got[7:41], c[7:41])
    dg.dg_route_balance_backward(x2.cuda(), dev(counts), dev(starts), None, None, out, k)
    assert (out[:7] == 0).all() and (out[41:] == 0).all()


def test_starts_out_of_range_are_cut_off(dg):
    T, E, k = 33, 16, 2
    _, x, ids, _ = problem(4, T, E, k, 0, "float32")
    far = np.array([-5, 10, 2 ** 31 - 1], dtype=np.int32)
    near = np.array([0, 10, T], dtype=np.int32)
    for a, b in zip(forward(dg, x, ids, far, "sigmoid"), forward(dg, x, ids, near, "sigmoid")):
        assert np.array_equal(a, b)


def test_small_workspace_and_many_sequences(dg):
    """With room for a few sums only, sequences go out in several launches: the same results."""
    T, E, k, S = 700, 30, 3, 150
    _, x, ids, starts = problem(9, T, E, k, S, "bfloat16")
    want = forward(dg, x, ids, starts, "sigmoid")
    stream = torch.cuda.Stream()
    ws = torch.zeros(256 + 9 * 32 * 8, dtype=torch.uint8, device="cuda")
    dg.dg_bind_stream_workspace(stream, ws)
    try:
        with torch.cuda.stream(stream):
            got = forward(dg, x, ids, starts, "sigmoid")
    finally:
        dg.dg_bind_stream_workspace(stream, None)
    assert np.array_equal(got[1], want[1])
    assert np.all(np.abs(got[0] - want[0]) <= (E + 160) * UNIT * want[0])


def test_the_same_bits_from_run_to_run(dg):
    _, x, ids, starts = problem(11, 5000, 160, 8, 3, "float32")
    a, b = (forward(dg, x, ids, starts, "sigmoid") for _ in range(2))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


ORDER = [
    # T, sequences: several per chunk of 64 tokens, one over many chunks, ends at the chunks' own ends
    (640, [0, 64, 128, 640]), (640, [0, 1, 2, 3, 63, 64, 65, 127, 128, 129, 640]), (3000, [5, 5, 5, 1999, 2000, 2001, 2999]),
    (4096, [0, 4096]), (4097, [0, 0, 4097, 4097]), (40000, [0, 13, 30000, 39999]),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [60, 256, 400, 1000])
@pytest.mark.parametrize("case", ORDER, ids=lambda c: f"{c[0]}-{len(c[1]) - 1}")
def test_sequences_across_chunks(dg, case, E, score):
    T, starts = case
    print(f"case: balance of {T} tokens in {len(starts) - 1} sequences, {E} experts, {score}", flush=True)
    T = T if E < 400 else min(T, 5000)
    starts = np.minimum(starts, T).astype(np.int32)
    _, x, ids, _ = problem(T + E, T, E, 5, 0, "bfloat16", masked=0.02)
    loss, counts = forward(dg, x, ids, starts, score)
    want, n = layer.balance(x.float().numpy(), ids, starts, score)
    assert np.array_equal(counts, n)
    # a lane adds up to T / 256 / 32 tokens by itself, 32 lanes' sums and then fp64
    assert np.all(np.abs(loss - want) <= (E + 160 + T / 2048) * UNIT * want)
    if T <= 4097:
        out = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
        dg.dg_route_balance_backward(x.cuda(), dev(counts), dev(starts), None, None, out, 5, score=score)
        want, mag = layer.balance_backward(x.float().numpy(), counts, starts, None, None, 5, score)
        got = out.double().cpu().numpy()
        bound = HALF["bfloat16"] * np.abs(want) + (E + 33) * UNIT * mag + 1e-37
        assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())


def test_counts_of_other_gpus(dg):
    """The gradient takes counts as they are given: those of a whole job's tokens, up to the ends of int32."""
    T, E, k = 20, 16, 4
    rng, x, ids, _ = problem(6, T, E, k, 0, "float32")
    counts = rng.integers(0, 2 ** 31 - 1, (1, E)).astype(np.int32)
    counts[0, :2] = 0, 2 ** 31 - 1
    out = torch.empty(T, E, device="cuda")
    for score in ("softmax", "sigmoid"):
        dg.dg_route_balance_backward(x.cuda(), dev(counts), None, None, None, out, k, score=score)
        want, mag = layer.balance_backward(x.numpy(), counts, None, None, None, k, score)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= UNIT * np.abs(want) + (E + 33) * UNIT * mag)
