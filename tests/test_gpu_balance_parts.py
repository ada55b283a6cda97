"""The balance loss in its two kernels: sequences that go out in several launches, a
workspace without room, graphs, and long sequences.

Bounds as in test_gpu_balance.py, with the fp32 sums over tokens as they are here: a
chunk of c tokens is added up in 32 runs (16 from 257 experts on, 8 from 513), and these
one after the other; all else is fp64."""
import numpy as np
import pytest
import torch

from oracle import layer
from tests.test_gpu_balance import UNIT, forward, problem
from tests.workspaces import Bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    yield m
    torch.cuda.empty_cache()


def runs(E):
    return 32 if E <= 256 else 16 if E <= 512 else 8


def units(E, chunk):
    """of 2^-24: the share (E + 16), the run's tokens, the runs, rounding of the result"""
    return E + 16 + -(-chunk // runs(E)) + runs(E) + 2


def room_for(rows, E):
    """Bytes of `rows` sums and counts of E experts."""
    return rows * -(-E // 4) * 32


# T, E, top_k, sequences, rows of sums that there is room for (half of them at most for the chunks, the others for the
# sequences of one launch), type
PARTS = [
    (6000, 30, 3, 150, 12, "bfloat16"), (6000, 30, 3, 150, 2, "float32"), (9001, 8, 2, 7, 5, "float32"),
    (3000, 256, 8, 40, 5, "bfloat16"), (2500, 400, 4, 33, 9, "float32"), (1000, 1000, 8, 20, 3, "bfloat16"),
    (7000, 64, 6, 3000, 700, "float32"), (5000, 60, 4, 1, 2, "float32"),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", PARTS, ids=lambda c: "-".join(map(str, c)))
def test_sequences_in_several_launches(dg, case, score):
    T, E, k, S, rows, dtype = case
    print(f"case: balance in parts {case} {score}", flush=True)
    assert T * max(64, E) > 32768 * min(S, 4)                    # beyond what one workgroup per sequence takes
    _, x, ids, starts = problem(T + E + S, T, E, k, S, dtype, masked=0.03 if E > 8 else 0.0)
    with Bound(dg, room_for(rows, E)):
        loss, counts = forward(dg, x, ids, starts, score, scale=0.5)
    want, n = layer.balance(x.float().numpy(), ids, starts, score, scale=0.5)
    assert np.array_equal(counts, n)
    chunk = -(-T // (rows // 2)) + 64
    assert np.all(np.abs(loss - want) <= units(E, chunk) * UNIT * want)


def test_sequences_that_begin_and_end_with_chunks_and_launches(dg):
    """With room for 8 sums: 4 chunks of 1504 tokens, 4 sequences to a launch."""
    T, E, k = 6016, 40, 4
    _, x, ids, _ = problem(1, T, E, k, 0, "float32")
    for starts in ([0, 1504, 3008, 4512, 6016], [0, 0, 0, 0, 1504, 1504, 1505, 6016, 6016], [3, 1503, 1504, 4000, 4512, 4513, 6015],
                   [0, 6016], [1504] * 9 + [1600], list(range(0, 6017, 16))):
        starts = np.array(starts, dtype=np.int32)
        with Bound(dg, room_for(8, E)):
            loss, counts = forward(dg, x, ids, starts, "softmax")
        want, n = layer.balance(x.numpy(), ids, starts, "softmax")
        assert np.array_equal(counts, n), starts
        assert np.all(np.abs(loss - want) <= units(E, 1504) * UNIT * want), starts


def test_no_room(dg):
    _, x, ids, starts = problem(2, 6000, 30, 3, 5, "float32")
    with Bound(dg, room_for(1, 30)):
        with pytest.raises(dg.DGError, match="no room for the sums of 30 experts") as e:
            forward(dg, x, ids, starts, "softmax")
        assert e.value.status == -2
        few, n = forward(dg, x[:100], ids[:100], None, "softmax")             # one launch needs none
    want, m = layer.balance(x[:100].numpy(), ids[:100], None, "softmax")
    assert np.array_equal(n, m) and np.all(np.abs(few - want) <= units(30, 100) * UNIT * want)


@pytest.mark.parametrize("rows", [None, 12])
def test_two_kernels_in_a_graph(dg, rows):
    """Captured once, replayed with other inputs and starts, with eager calls between: the same bits, and the oracle's."""
    print(f"case: balance of two kernels under graph replay, rows={rows}", flush=True)
    T, E, k, S = 5000, 24, 3, 31
    logits = torch.empty(T, E, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    starts = torch.empty(S + 1, dtype=torch.int32, device="cuda")
    loss, counts = torch.empty(S, device="cuda"), torch.empty(S, E, dtype=torch.int32, device="cuda")
    grad = torch.empty_like(logits)

    def step():
        dg.dg_route_balance(logits, ids, starts, loss, counts, score="sigmoid")
        dg.dg_route_balance_backward(logits, counts, starts, loss, None, grad, k, score="sigmoid")

    def fill(seed):
        _, x, i, s = problem(seed, T, E, k, S, "float32", masked=0.02)
        logits.copy_(x)
        ids.copy_(torch.from_numpy(i))
        starts.copy_(torch.from_numpy(s))
        torch.cuda.synchronize()
        return x, i, s

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    bound = Bound(dg, room_for(rows, E)) if rows else None
    if bound:
        dg.dg_bind_stream_workspace(bound.stream, bound.ws)
    try:
        with torch.cuda.graph(graph, stream=bound.stream if bound else torch.cuda.Stream()):
            step()
    finally:
        if bound:
            dg.dg_bind_stream_workspace(bound.stream, None)
    for rep in range(4):
        x, i, s = fill(rep + 1)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (loss, counts, grad)]
        step()
        torch.cuda.synchronize()
        want, n = layer.balance(x.numpy(), i, s, "sigmoid")
        assert np.array_equal(got[1].cpu().numpy(), n)
        assert np.all(np.abs(got[0].double().cpu().numpy() - want) <= units(E, T // 6 + 64) * UNIT * want)
        if not rows:                             # (the eager calls take other chunks than with the small workspace)
            assert torch.equal(got[0], loss) and torch.equal(got[2], grad), rep
        assert torch.equal(got[1], counts), rep


@pytest.mark.parametrize("E", [60, 300, 1000])
def test_long_sequences(dg, E):
    """A sequence of a million tokens with equal shares, which all round alike when they are added up, and one of other
    shares behind it: off by less than (E + 160 + T / 4096) * 2^-24."""
    print(f"case: balance of 1000003 tokens of {E} experts", flush=True)
    T, k, tail = 1000003, 2, 70000
    logits = torch.zeros(T, E, device="cuda")
    own = torch.randn(tail, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(E))
    logits[T - tail:] = own
    ids = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).view(T, k)
    starts = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    loss, counts = torch.empty(2, device="cuda"), torch.empty(2, E, dtype=torch.int32, device="cuda")
    dg.dg_route_balance(logits, ids, starts, loss, counts)
    torch.cuda.synchronize()
    n = torch.stack([torch.bincount(i.flatten().long(), minlength=E) for i in (ids[:T - tail], ids[T - tail:])])
    assert torch.equal(counts.long(), n)
    p = torch.stack([torch.full((E,), (T - tail) / E, device="cuda", dtype=torch.double), torch.softmax(own.double(), 1).sum(0)])
    length = torch.tensor([T - tail, tail], device="cuda", dtype=torch.double)
    want = E / (k * length ** 2) * (n * p).sum(1)
    assert bool(((loss.double() - want).abs() <= (E + 160 + T / 4096) * UNIT * want).all()), (loss.double() / want - 1).tolist()
