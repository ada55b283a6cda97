"""The operators around the products together: the example layer against float64,
captured in a HIP graph whose inputs change between replays, and on two streams
at once with their own workspaces; and the same bits from run to run."""
import numpy as np
import pytest
import torch

import examples.moe_layer as moe
from oracle import around
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    m.dg_init()
    return m


@pytest.mark.parametrize("T", [1, 7, 300, 1000])
def test_example_layer(dg, T):
    print(f"case: example layer, {T} tokens", flush=True)
    far = moe.check(T=T, seed=T)
    # two e4m3 operands: each value is off by up to 2^-4 of itself, 0.026 in the
    # root mean square over a binade; two of them 0.037, averaged over K = 512
    assert far["d"] < 0.05 and far["gradient of the experts"] < 0.05
    # against float64 from the layer's own gradient of the weights: fp32 rounding only
    assert far["gradient of the logits"] < 0.08
    assert far["served, contiguous"] == 0.0
    # the masked product takes other tiles: fp32 sums in another order, then bf16
    assert far["served, masked"] < 2.0 ** -8


def test_serving_step_in_a_graph(dg):
    print("case: serving step under graph replay, inputs changed between replays", flush=True)
    layer, w, g = moe.make(seed=3)
    H, L = 512, 5
    x, ids = moe.tokens(g, 40, H, L)
    for max_m in (40, None):
        eager = lambda: layer.serve(x, ids, max_m=max_m)
        eager()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            out = eager()
        for rep in range(4):
            nx, nids = moe.tokens(g, 40, H, L)
            x.copy_(nx)
            ids.copy_(nids)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert torch.equal(got, eager()), (max_m, rep)
            torch.cuda.synchronize()


def test_training_calls_in_a_graph(dg):
    print("case: gradients and large layouts under graph replay", flush=True)
    rng = np.random.default_rng(0)
    T, E, k, N = 5000, 24, 4, 256
    logits = torch.empty(T, E, device="cuda")
    ids, weights = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    M = dg.dg_m_grouped_rows_bound(T * k, E)
    i32 = dict(dtype=torch.int32, device="cuda")
    layout, row_of, slot_of, counts = torch.empty(M, **i32), torch.empty(T, k, **i32), torch.empty(M, **i32), torch.empty(E, **i32)
    x = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    a, sfa = torch.zeros(M, N, dtype=torch.uint8, device="cuda"), torch.zeros(N // 128, M, device="cuda")
    ka, ksf = torch.zeros(M, N, dtype=torch.uint8, device="cuda"), torch.zeros(M // 128, N, device="cuda")
    rows = torch.randn(M, N, device="cuda").to(torch.bfloat16)
    gw, gl = torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")

    def step():
        dg.dg_route_topk(logits, None, ids, weights)
        dg.dg_m_grouped_layout_contiguous(ids, 0, layout, row_of, slot_of, counts)
        dg.dg_m_grouped_scatter_fp8_contiguous(x, weights, row_of, slot_of, a, sfa)
        dg.dg_k_grouped_scatter_fp8(x, weights, slot_of, k, ka, ksf)
        dg.dg_m_grouped_gather_weight_grad(rows, row_of, x, gw)
        dg.dg_route_topk_backward(logits, ids, gw, gl)

    outs = [ids, weights, layout, row_of, slot_of, counts, a, sfa, ka, ksf, gw, gl]

    def fill():
        logits.copy_(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))
        x.copy_(torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)))
        a.zero_()
        sfa.zero_()

    fill()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for rep in range(3):
        fill()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        a.zero_()
        sfa.zero_()
        step()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(got, outs)):
            assert torch.equal(p, q), (rep, i)


def test_two_streams_with_their_own_workspaces(dg):
    print("case: layouts, scatters and adapters on two streams at once", flush=True)
    rng = np.random.default_rng(5)
    T, G, k, K, L, R, N = 9000, 40, 4, 256, 6, 32, 136
    M = dg.dg_m_grouped_rows_bound(T * k, G)
    i32 = dict(dtype=torch.int32, device="cuda")
    jobs, streams, spaces = [], [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        ids = np.stack([rng.permutation(G)[:k] for _ in range(T)]).astype(np.int32)
        x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
        la = torch.from_numpy(rng.standard_normal((L, R, K)).astype(np.float32)).to(torch.bfloat16).cuda()
        lb = torch.from_numpy(rng.standard_normal((L, N, R)).astype(np.float32)).to(torch.bfloat16).cuda()
        aid = dev(rng.integers(-1, L, T).astype(np.int32))
        jobs.append(dict(ids=ids, d_ids=dev(ids), x=x, la=la, lb=lb, aid=aid,
                         maps=(torch.empty(M, **i32), torch.empty(T, k, **i32), torch.empty(M, **i32), torch.empty(G, **i32)),
                         a=torch.zeros(M, K, dtype=torch.uint8, device="cuda"), sfa=torch.zeros(K // 128, M, device="cuda"),
                         d=torch.empty(T, N, dtype=torch.bfloat16, device="cuda")))
        spaces.append(torch.empty(4 << 20, dtype=torch.uint8, device="cuda"))

    def run(j, stream):
        dg.dg_m_grouped_layout_contiguous(j["d_ids"], 0, *j["maps"], stream=stream)
        dg.dg_m_grouped_scatter_fp8_contiguous(j["x"], None, j["maps"][1], j["maps"][2], j["a"], j["sfa"], stream=stream)
        dg.dg_lora_bf16_nt(j["x"], j["la"], j["lb"], None, j["aid"], None, j["d"], stream=stream)

    want = []
    for j in jobs:
        run(j, None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (*j["maps"], j["a"], j["sfa"], j["d"])])
        for got, ref in zip(j["maps"], around.layout_contiguous(j["ids"], 0, G, M)):
            assert np.array_equal(got.cpu().numpy(), ref)
        for t in (*j["maps"], j["a"], j["sfa"], j["d"]):
            t.zero_()
    torch.cuda.synchronize()
    try:
        for s, w in zip(streams, spaces):
            dg.dg_bind_stream_workspace(s, w)
        for _ in range(10):
            for j, s in zip(jobs, streams):
                run(j, s)
        torch.cuda.synchronize()
        for j, ref in zip(jobs, want):
            for p, q in zip((*j["maps"], j["a"], j["sfa"], j["d"]), ref):
                assert torch.equal(p, q)
    finally:
        for s in streams:
            dg.dg_bind_stream_workspace(s, None)


def test_adapters_with_small_workspaces(dg):
    # the tokens go through in as many parts as the workspace needs, with the same
    # bound on the error; none at all is refused
    print("case: adapters with bound workspaces of several sizes", flush=True)
    rng = np.random.default_rng(9)
    T, L, R, N, K = 700, 4, 24, 70, 512
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16)
    a = torch.from_numpy(rng.standard_normal((L, R, K)).astype(np.float32) * K ** -0.5).to(torch.bfloat16)
    b = torch.from_numpy(rng.standard_normal((L, N, R)).astype(np.float32) * 0.1).to(torch.bfloat16)
    ids = rng.integers(-1, L, T).astype(np.int32)
    ref, mag = around.lora(x.float().numpy(), a.float().numpy(), b.float().numpy(), None, ids, None)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 + (K + R) * 2.0 ** -24) * mag + 1e-37
    st = torch.cuda.Stream()
    xd, ad, bd, idd = x.cuda(), a.cuda(), b.cuda(), dev(ids)
    d = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for room in (16 * R * 4, 40 * R * 4 + 100, 4096, 1 << 17):
        d.fill_(float("nan"))
        torch.cuda.synchronize()
        buf = torch.empty(256 + room if room < 4096 else 256 + 4096 + room, dtype=torch.uint8, device="cuda")
        dg.dg_bind_stream_workspace(st, buf)
        try:
            dg.dg_lora_bf16_nt(xd, ad, bd, None, idd, None, d, stream=st)
            st.synchronize()
        finally:
            dg.dg_bind_stream_workspace(st, None)
        assert np.all(np.abs(d.float().cpu().numpy() - ref) <= bound), room
    buf = torch.empty(256, dtype=torch.uint8, device="cuda")
    dg.dg_bind_stream_workspace(st, buf)
    try:
        with pytest.raises(dg.DGError, match="no room") as e:
            dg.dg_lora_bf16_nt(xd, ad, bd, None, idd, None, d, stream=st)
        assert e.value.status == -2
    finally:
        dg.dg_bind_stream_workspace(st, None)


def test_same_bits_from_run_to_run(dg):
    print("case: repeated calls give the same bits", flush=True)
    rng = np.random.default_rng(12)
    T, L, R, N, K = 600, 3, 48, 200, 1024
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    a = torch.from_numpy(rng.standard_normal((L, R, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    b = torch.from_numpy(rng.standard_normal((L, N, R)).astype(np.float32)).to(torch.bfloat16).cuda()
    rows = torch.from_numpy(rng.standard_normal((900, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    at = dev(rng.integers(-1, 900, (T, 5)).astype(np.int32))
    w = dev(rng.standard_normal((T, 5)).astype(np.float32))
    for t in (60, T):
        ids = dev(rng.integers(-1, L, t).astype(np.int32))
        first = None
        for _ in range(4):
            d = torch.empty(t, N, dtype=torch.bfloat16, device="cuda")
            dg.dg_lora_bf16_nt(x[:t], a, b, None, ids, None, d)
            e = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
            dg.dg_m_grouped_gather(rows, at, w, None, e)
            gw = torch.empty(T, 5, device="cuda")
            dg.dg_m_grouped_gather_weight_grad(rows, at, e, gw)
            torch.cuda.synchronize()
            if first is None:
                first = (d, e, gw)
            assert all(torch.equal(p, q) for p, q in zip(first, (d, e, gw)))
