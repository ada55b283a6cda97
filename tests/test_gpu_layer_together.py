"""The balance loss, the 4-bit products and the gradients' clipping together, as a
layer is trained and served: the example layer, HIP graphs whose inputs change
between replays, two streams at once with their own workspaces."""
import numpy as np
import pytest
import torch

import examples.moe_layer as moe
from oracle import layer as oracle_layer
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    m.dg_init()
    return m


@pytest.mark.parametrize("T", [1, 7, 300])
def test_example_layer(dg, T):
    print(f"case: example layer trained and served on 4-bit weights, {T} tokens", flush=True)
    far = moe.check(T=T, seed=T + 20)
    # each value: y rounded to bf16 twice, rows and d once, 2^-8 at most each
    assert far["served, 4-bit"] < 4 * 2.0 ** -8
    # fp32 rounding only (tests of the operators themselves have the bounds): shares of
    # 16 experts within 32 units of 2^-24, sums within a few more
    assert far["balance loss"] < 200 * 2.0 ** -24
    assert far["gradient with the balance loss"] < 200 * 2.0 ** -24
    assert far["norm"] < 2 * 2.0 ** -24


def test_training_step_clips(dg):
    print("case: a training step with its gradients clipped", flush=True)
    lay, w, g = moe.make(seed=4)
    x, ids = moe.tokens(g, 200, 512, 5)
    grad_d = torch.randn(200, 512, device="cuda", generator=g).to(torch.bfloat16)
    starts = torch.tensor([0, 50, 50, 180], dtype=torch.int32, device="cuda")    # an empty sequence, 20 tokens of padding
    _, free, norm, loss, counts = lay.train_step(x, ids, grad_d, starts, max_norm=1e30)
    _, clipped, again, _, _ = lay.train_step(x, ids, grad_d, starts, max_norm=0.25)
    assert torch.equal(norm, again) and float(norm) > 0.25
    f = 0.25 / (float(norm) + 1e-6)
    for k in free:
        assert ((clipped[k].double() - free[k].double() * f).abs() <= 4 * 2.0 ** -24 * free[k].double().abs() * f + 1e-45).all()
    assert float(loss[1]) == 0.0 and int(counts[1].sum()) == 0 and int(counts.sum()) == 180 * lay.top_k
    total = sum(v.double().square().sum() for v in clipped.values()).sqrt()
    assert abs(float(total) - 0.25) < 1e-5


def test_serving_step_in_a_graph(dg):
    print("case: 4-bit serving step under graph replay, inputs changed between replays", flush=True)
    lay, w, g = moe.make(seed=6)
    for T in (1, 6, 40):
        x, ids = moe.tokens(g, T, 512, 5)
        lay.serve_few(x, ids)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            out = lay.serve_few(x, ids)
        for rep in range(4):
            nx, nids = moe.tokens(g, T, 512, 5)
            x.copy_(nx)
            ids.copy_(nids)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert torch.equal(got, lay.serve_few(x, ids)), (T, rep)
            torch.cuda.synchronize()


def test_all_calls_in_a_graph(dg):
    """Every new call captured once and replayed with other inputs: the same bits as the eager calls."""
    print("case: balance, 4-bit products by lists and clipping under graph replay", flush=True)
    rng = np.random.default_rng(0)
    T, E, k, N, K = 1500, 24, 3, 72, 256
    logits = torch.empty(T, E, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    starts = torch.empty(8, dtype=torch.int32, device="cuda")
    loss, counts = torch.empty(7, device="cuda"), torch.empty(7, E, dtype=torch.int32, device="cuda")
    grad = torch.empty_like(logits)
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    b = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    sc = torch.rand(E, K // 32, N, device="cuda")
    rows = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda")
    norm = torch.empty(1, device="cuda")
    outs = [torch.empty_like(grad), torch.empty_like(rows)]

    def step():
        dg.dg_route_balance(logits, ids, starts, loss, counts, score="sigmoid")
        dg.dg_route_balance_backward(logits, counts, starts, loss, None, grad, k, score="sigmoid")
        dg.dg_m_grouped_bf16_int4_gemv_nt_topk(x, ids, 2, b[:20], sc[:20], None, None, rows)
        dg.dg_grad_norm([grad, rows], norm)
        dg.dg_grad_clip([grad, rows], outs, norm, 0.5)

    def fill():
        logits.copy_(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))
        ids.copy_(torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)))
        starts.copy_(torch.from_numpy(np.sort(rng.integers(0, T + 1, 8)).astype(np.int32)))
        x.copy_(torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)))

    fill()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for rep in range(4):
        fill()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (loss, counts, grad, rows, norm, *outs)]
        step()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(got, (loss, counts, grad, rows, norm, *outs))):
            assert torch.equal(p, q), (rep, i)


def test_two_streams_with_their_own_workspaces(dg):
    print("case: balance, 4-bit products by lists and norms on two streams at once", flush=True)
    rng = np.random.default_rng(5)
    T, E, k, N, K = 3000, 40, 2, 48, 128
    jobs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(4 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for _ in range(2):
        j = dict(logits=dev(rng.standard_normal((T, E)).astype(np.float32)),
                 ids=dev(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)),
                 starts=dev(np.sort(rng.integers(0, T + 1, 5)).astype(np.int32)), loss=torch.empty(4, device="cuda"),
                 counts=torch.empty(4, E, dtype=torch.int32, device="cuda"),
                 x=torch.randn(T, K, device="cuda").to(torch.bfloat16),
                 b=torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda"),
                 sfb=torch.full((E, K // 128, N), 0x7E7D7F7C, dtype=torch.int32, device="cuda"),
                 rows=torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda"), norm=torch.empty(1, device="cuda"))
        jobs.append(j)

    def run(j, stream):
        dg.dg_route_balance(j["logits"], j["ids"], j["starts"], j["loss"], j["counts"], stream=stream)
        dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(j["x"], j["ids"], 0, j["b"], j["sfb"], None, j["rows"], stream=stream)
        dg.dg_grad_norm([j["logits"], j["rows"]], j["norm"], stream=stream)

    outs = ("loss", "counts", "rows", "norm")
    want = []
    for j in jobs:
        run(j, None)
        torch.cuda.synchronize()
        want.append([j[o].clone() for o in outs])
        for o in outs:
            j[o].zero_()
    torch.cuda.synchronize()
    try:
        for s, w in zip(streams, spaces):
            dg.dg_bind_stream_workspace(s, w)
        for _ in range(10):
            for j, s in zip(jobs, streams):
                run(j, s)
        torch.cuda.synchronize()
        for j, ref in zip(jobs, want):
            for o, r in zip(outs, ref):
                assert torch.equal(j[o], r), o
    finally:
        for s in streams:
            dg.dg_bind_stream_workspace(s, None)


def test_the_few_products_agree_with_the_fp4_products(dg):
    """The same weights through the FP8 x FP4 product, on activations that e4m3 holds exactly: the same results but
    for fp32 sums in another order."""
    print("case: 4-bit products against the FP8 x FP4 product", flush=True)
    rng = np.random.default_rng(2)
    M, N, K = 33, 200, 512
    q = torch.from_numpy(rng.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5], (M, K)).astype(np.float32))
    b = dev(rng.integers(0, 256, (N, K // 2), dtype=np.uint8))
    sfb = dev(rng.integers(122, 128, (K // 128, N, 4), dtype=np.uint8).view(np.int32).reshape(K // 128, N))
    d8, d16 = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.dg_fp8_fp4_gemm_nt(q.to(torch.float8_e4m3fn).cuda(), torch.ones(K // 128, M, device="cuda"), b, sfb, None, d8)
    dg.dg_bf16_fp4_gemv_nt(q.to(torch.bfloat16).cuda(), b, sfb, None, d16)
    w = oracle_layer.fp4_weights(b.cpu().numpy(), sfb.cpu().numpy())
    ref, mag = oracle_layer.gemv(q.double().numpy(), w, None)
    for d in (d8, d16):
        err = np.abs(d.double().cpu().numpy() - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag)
