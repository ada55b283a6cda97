"""The calls through the native side of the binding: taken wherever the arguments fit, with the same bits as through
the checks in Python, and the library's refusals raised in the same way."""
import pytest
import torch

import moe_grouped_gemm_nt_amd._lib as lib

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    return m


def calls(dg, seed=0):
    """name -> (call, outputs): every call of the native side, with strided rows and left-out tensors among them"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    def f(*s):
        return torch.randn(*s, device="cuda", generator=g)
    def i(lo, hi, *s, t=torch.int32):
        return torch.randint(lo, hi, s, device="cuda", generator=g, dtype=t)
    T, E, k, N, K, G = 7, 24, 3, 40, 256, 5
    logits, ids = f(T, E).to(bf), f(T, E).topk(k).indices.int()
    starts = torch.tensor([0, 3, 7], device="cuda", dtype=torch.int32)
    loss, counts, back = f(2), i(0, 4, 2, E), f(T, E).to(bf)
    x = f(T, 2 * K).to(bf)[:, :K]
    b, wide = i(0, 256, G, N, K // 2, t=torch.uint8), f(T, N + 8).to(bf)
    sfb = (i(118, 130, G, K // 128, N, 4, t=torch.uint8)).view(torch.int32).squeeze(-1).contiguous()
    scales, zeros = f(G, K // 64, N), i(0, 16, G, K // 64, N, t=torch.uint8)
    d, few, own = f(T, N).to(bf), f(T * k, N).to(bf), i(0, G + 1, T, k)
    grads, norm = [f(5, 3), f(4097).to(bf)], f(1)
    outs = [torch.empty_like(t) for t in grads]
    return {
        "dg_route_balance": (lambda s=None: dg.dg_route_balance(logits, ids, starts, loss, counts, "sigmoid", 2, s),
                             [loss, counts]),
        "dg_route_balance_backward": (lambda s=None: dg.dg_route_balance_backward(
            logits, ids.new_ones(2, E), starts, None, back, back, k, stream=s), [back]),
        "dg_bf16_fp4_gemv_nt": (lambda s=None: dg.dg_bf16_fp4_gemv_nt(x, b[0], sfb[0], wide[:, 8:], d, s), [d]),
        "dg_bf16_int4_gemv_nt": (lambda s=None: dg.dg_bf16_int4_gemv_nt(
            x, b[1], scales[1].to(bf), None, None, wide[:, :N], s), [wide]),
        "dg_m_grouped_bf16_fp4_gemv_nt_topk": (lambda s=None: dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(
            x, own, 1, b, sfb, None, few, s), [few]),
        "dg_m_grouped_bf16_int4_gemv_nt_topk": (lambda s=None: dg.dg_m_grouped_bf16_int4_gemv_nt_topk(
            x, own, 0, b, scales, zeros, None, few, s), [few]),
        "dg_grad_norm": (lambda s=None: dg.dg_grad_norm(grads, norm, s), [norm]),
        "dg_grad_clip": (lambda s=None: dg.dg_grad_clip(tuple(grads), outs, norm, 1, s), outs),
    }


def test_both_sides_give_the_same_bits(dg, monkeypatch):
    fast, taken = lib._fast, []
    def counted(fn, *args):
        taken.append((fn, fast(fn, *args)))
        return taken[-1][1]
    bits = []
    for here in (counted, lambda *a: False):
        monkeypatch.setattr(lib, "_fast", here)
        for name, (call, outputs) in calls(dg).items():
            call()
            bits.append([o.clone() for o in outputs])
    assert [n for n, done in taken if done] == list(calls(dg))
    half = len(bits) // 2
    for a, b in zip(bits[:half], bits[half:]):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b))


@pytest.mark.parametrize("kind", ["raw", "object"])
def test_a_stream_given(dg, kind):
    for name in calls(dg, 1):                    # (inputs of its own for each: the norm is one call's output, another's input)
        (call, outputs), (want_call, want) = calls(dg, 1)[name], calls(dg, 1)[name]
        want_call()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        call(other.cuda_stream if kind == "raw" else other)
        other.synchronize()
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(outputs, want)), name


def test_refusals_of_the_library_are_raised(dg):
    x = torch.zeros(4, 2048, device="cuda")
    ids, loss = torch.zeros(4, 2, device="cuda", dtype=torch.int32), torch.zeros(1, device="cuda")
    with pytest.raises(dg.DGError, match="1024"):              # more experts than a router may have
        dg.dg_route_balance(x, ids, None, loss, torch.zeros(1, 2048, device="cuda", dtype=torch.int32))
    g = torch.zeros(64, device="cuda")
    with pytest.raises(dg.DGError, match="apart"):
        dg.dg_grad_clip([g[:32]], [g[16:48]], loss, 1.0)


def test_two_host_threads(dg):
    """Calls from two threads, each on its own stream with its own workspace, give the bits of calls in turn."""
    import threading
    results, errors = [None, None], []

    def work(t):
        try:
            stream = torch.cuda.Stream()
            ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
            with torch.cuda.stream(stream):
                dg.dg_bind_stream_workspace(stream, ws)
                try:
                    made = [calls(dg, t)[name] for name in calls(dg, t)]
                    for call, _ in made * 20:
                        call()
                    results[t] = [o.clone() for _, outputs in made for o in outputs]
                    stream.synchronize()
                finally:
                    dg.dg_bind_stream_workspace(stream, None)
        except Exception as e:                                    # (shown by the assertion below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for t in (0, 1):
        made = [calls(dg, t)[name] for name in calls(dg, t)]
        for call, _ in made * 20:
            call()
        want = [o for _, outputs in made for o in outputs]
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(results[t], want))


def test_captured_and_replayed(dg):
    """The calls in one graph, with eager ones of the same buffers between the replays."""
    made = [calls(dg, 2)[name] for name in calls(dg, 2)]
    eager = [calls(dg, 2)[name] for name in calls(dg, 2)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for call, _ in made:
            call()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        for call, _ in eager:
            call()
        torch.cuda.synchronize()
        for (_, a), (_, b) in zip(made, eager):
            assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b))
