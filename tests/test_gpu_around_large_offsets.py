"""Offsets beyond 2^31 elements and 2^32 bytes in every operand of the operators
around the products that can be that large: values at the far end of buffers of
4 to 9 GB, against the fp64 oracle on the rows concerned."""
import numpy as np
import pytest
import torch

import oracle
from oracle import around
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    yield m
    torch.cuda.empty_cache()


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def test_gather_and_its_weight_gradient(dg):
    print("case: gather from 300000 x 7500 rows", flush=True)
    rng = np.random.default_rng(0)
    M, N, T = 300000, 7500, 3
    rows = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    far = np.array([M - 1, M - 2, 143166, 5])        # 143166 * 7500 * 2 is just beyond 2^31
    v = bf16(rng, 4, N)
    rows[torch.from_numpy(far).cuda()] = v.cuda()
    at = far[[[0, 1], [2, 3], [3, 0]]].astype(np.int32)
    d = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_gather(rows, dev(at), None, None, d)
    gw = torch.empty(T, 2, device="cuda")
    dg.dg_m_grouped_gather_weight_grad(rows, dev(at), d, gw)
    torch.cuda.synchronize()
    near = np.array([[0, 1], [2, 3], [3, 0]], dtype=np.int32)
    ref, mag = around.gather(v.float().numpy(), near, None, None)
    assert np.all(np.abs(d.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * mag)
    ref, mag = around.gather_weight_grad(v.float().numpy(), near, d.float().cpu().numpy())
    assert np.all(np.abs(gw.cpu().numpy() - ref) <= N * 2.0 ** -24 * mag)


def test_scatters(dg):
    print("case: scatter into 600064 x 7168 rows", flush=True)
    rng = np.random.default_rng(1)
    M, K = 600064, 7168
    x = bf16(rng, 2, K)
    row_of = torch.tensor([[M - 1, 7], [M - 64, 299593]], dtype=torch.int32)       # 299593 * 7168 is beyond 2^31
    slot_of = torch.full((M,), -1, dtype=torch.int32)
    slot_of[row_of.view(-1).long()] = torch.arange(4, dtype=torch.int32)
    a = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(K // 128, M, device="cuda")
    dg.dg_m_grouped_scatter_fp8_contiguous(x.cuda(), None, row_of.cuda(), slot_of.cuda(), a, sfa)
    torch.cuda.synchronize()
    live = row_of.view(-1).long().cuda()
    got = oracle.decode_e4m3(a[live].cpu().numpy()).reshape(4, K // 128, 128) * sfa[:, live].t().cpu().numpy()[:, :, None]
    want = x.float().numpy()[[0, 0, 1, 1]].reshape(4, K // 128, 128)
    amax = np.abs(want).max(axis=2, keepdims=True)
    assert np.all(np.abs(got - want) <= amax * (16.0 / 448.0 + 1e-6))              # half of the widest step
    assert int((a != 0).any(1).sum()) == 4 and int((sfa != 0).any(0).sum()) == 4
    ka = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    ksf = torch.zeros(M // 128, K, device="cuda")
    dg.dg_k_grouped_scatter_fp8(x.cuda(), None, slot_of.cuda(), 2, ka, ksf)
    torch.cuda.synchronize()
    block = torch.div(live, 128, rounding_mode="floor")
    got = oracle.decode_e4m3(ka[live].cpu().numpy()) * ksf[block].cpu().numpy()
    want = x.float().numpy()[[0, 0, 1, 1]]
    assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * 1.001 + 1e-6)
    assert int((ka != 0).any(1).sum()) == 4


def test_router_and_its_gradient(dg):
    print("case: router over 4500000 x 512 logits", flush=True)
    rng = np.random.default_rng(2)
    T, E, k = 4500000, 512, 2
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    far = [T - 1, T - 2, 4194304, 3]                   # 4194304 * 512 = 2^31
    v = bf16(rng, 4, E)
    logits[torch.tensor(far, device="cuda")] = v.cuda()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    dg.dg_route_topk(logits, None, ids, w)
    torch.cuda.synchronize()
    ref_ids, ref_w, _ = around.route(v.float().numpy(), None, k, "softmax")
    assert np.array_equal(ids[far].cpu().numpy(), ref_ids)
    assert np.all(np.abs(w[far].cpu().numpy() - ref_w) <= 5e-6 * ref_w)
    assert torch.equal(ids[10:4194304].cpu(), torch.tensor([[0, 1]], dtype=torch.int32).expand(4194294, 2))
    gl = torch.empty_like(logits)
    dg.dg_route_topk_backward(logits, ids, w, gl)
    torch.cuda.synchronize()
    ref = around.route_backward(v.float().numpy(), ref_ids, w[far].cpu().numpy(), "softmax", True, 1.0)
    assert np.all(np.abs(gl[far].float().cpu().numpy() - ref) <= 1e-5 + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("T", [5, 300])
def test_adapters(dg, T):
    print(f"case: adapters of 1024 x 256 x 9216, {T} tokens", flush=True)
    rng = np.random.default_rng(3)
    L, R, K, N = 1024, 256, 9216, 40
    a = torch.zeros(L, R, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(L, N, R, dtype=torch.bfloat16, device="cuda")
    used = [L - 1, 911, 2]                             # 911 * 256 * 9216 is beyond 2^31
    va = (bf16(rng, 3, R, K).float() * K ** -0.5).to(torch.bfloat16)
    vb = bf16(rng, 3, N, R)
    a[torch.tensor(used, device="cuda")] = va.cuda()
    b[torch.tensor(used, device="cuda")] = vb.cuda()
    x = bf16(rng, T, K)
    near = rng.integers(0, 3, T)
    ids = np.array(used, dtype=np.int32)[near]
    d = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    dg.dg_lora_bf16_nt(x.cuda(), a, b, None, dev(ids), None, d)
    torch.cuda.synchronize()
    ref, mag = around.lora(x.float().numpy(), va.float().numpy(), vb.float().numpy(), None, near, None)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 + (K + R) * 2.0 ** -24) * mag + 1e-37
    assert np.all(np.abs(d.float().cpu().numpy() - ref) <= bound)
