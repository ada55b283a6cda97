"""What the operators around the products refuse, on the host and without a GPU:
through the C ABI (before any HIP call) and through the Python binding."""
import ctypes
import os

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as dg
from moe_grouped_gemm_nt_amd import _lib

INVALID, UNSUPPORTED, OK = _lib.DG_ERR_INVALID_ARG, _lib.DG_ERR_UNSUPPORTED, _lib.DG_OK
P = ctypes.c_void_p(0x100000)                  # aligned, never read: every call here ends on the host
ODD, BY2, BY4, BY8 = (ctypes.c_void_p(0x100000 + n) for n in (1, 2, 4, 8))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from moe_grouped_gemm_nt_amd import build
        build.build()
    return _lib.load()


def refused(lib, fn, base, status, needle, **change):
    args = dict(base, **change)
    assert getattr(lib, fn)(*args.values()) == status, (fn, change)
    if status != OK:
        assert needle in lib.dg_last_error().decode(), (fn, change, lib.dg_last_error())


ROUTE = dict(logits=P, type=0, bias=None, ids=P, w=P, T=4, E=64, k=8, score=1, G=8, kept=4, top=2, renorm=1,
             scale=1.0, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(logits=None), INVALID, "logits must not be NULL"), (dict(ids=None), INVALID, "topk_ids"),
    (dict(w=None), INVALID, "topk_weights"), (dict(type=2), INVALID, "logits_type"), (dict(score=5), INVALID, "score"),
    (dict(T=-1), INVALID, "negative"), (dict(E=0), INVALID, "top_k"), (dict(k=0), INVALID, "top_k"),
    (dict(k=65), INVALID, "top_k"), (dict(E=2048), UNSUPPORTED, "experts"),
    (dict(E=512, k=65, G=1, kept=1), UNSUPPORTED, "choices"), (dict(G=0), INVALID, "divide"),
    (dict(G=7), INVALID, "divide"), (dict(E=128, G=128), UNSUPPORTED, "num_groups"),
    (dict(kept=0), INVALID, "topk_groups"), (dict(kept=9), INVALID, "topk_groups"), (dict(top=3), INVALID, "group_top"),
    (dict(kept=1, k=9), INVALID, "exceeds the 8 experts"), (dict(logits=BY2), INVALID, "aligned"),
    (dict(bias=BY2), INVALID, "4-byte"), (dict(ids=ODD), INVALID, "4-byte"), (dict(w=BY2), INVALID, "4-byte"),
    (dict(T=0, logits=None, ids=None, w=None), OK, ""),
], ids=str)
def test_route(lib, change, status, needle):
    refused(lib, "dg_route_topk", ROUTE, status, needle, **change)


BACK = dict(logits=P, type=1, ids=P, gw=P, gx=P, T=4, E=64, k=8, score=0, renorm=1, scale=1.0, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(logits=None), INVALID, "NULL"), (dict(ids=None), INVALID, "NULL"), (dict(gw=None), INVALID, "NULL"),
    (dict(gx=None), INVALID, "NULL"), (dict(k=65), INVALID, "top_k"), (dict(E=1025, k=1), UNSUPPORTED, "experts"),
    (dict(gx=ODD), INVALID, "aligned"), (dict(ids=BY2), INVALID, "aligned"), (dict(score=-1), INVALID, "score"),
    (dict(T=0, logits=None, ids=None, gw=None, gx=None), OK, ""),
], ids=str)
def test_route_backward(lib, change, status, needle):
    refused(lib, "dg_route_topk_backward", BACK, status, needle, **change)


LAYOUT = dict(ids=P, T=4, k=2, first=0, G=8, M=128, layout=P, row=P, slot=P, counts=P, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(ids=None), INVALID, "NULL"), (dict(row=None), INVALID, "NULL"), (dict(slot=None), INVALID, "NULL"),
    (dict(layout=None), INVALID, "grouped_layout"), (dict(T=-1), INVALID, "T=-1"), (dict(k=0), INVALID, "top_k"),
    (dict(T=2**30, k=2), UNSUPPORTED, "choices"), (dict(G=0), INVALID, "num_groups"),
    (dict(G=1025), UNSUPPORTED, "num_groups"), (dict(M=100), INVALID, "multiple of 128"),
    (dict(M=-128), INVALID, "multiple of 128"), (dict(slot=BY2), INVALID, "4-byte"),
    (dict(counts=BY2), INVALID, "4-byte"), (dict(layout=ODD), INVALID, "4-byte"),
], ids=str)
def test_layout_contiguous(lib, change, status, needle):
    refused(lib, "dg_m_grouped_layout_contiguous", LAYOUT, status, needle, **change)


MASKED = dict(ids=P, T=4, k=2, first=0, G=8, m=16, masked=P, row=P, slot=P, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(ids=None), INVALID, "NULL"), (dict(masked=None), INVALID, "masked_m"), (dict(slot=None), INVALID, "NULL"),
    (dict(m=-1), INVALID, "max_m"), (dict(G=1024, m=2**22), UNSUPPORTED, "rows"), (dict(G=0), INVALID, "num_groups"),
    (dict(masked=BY2), INVALID, "4-byte"),
], ids=str)
def test_layout_masked(lib, change, status, needle):
    refused(lib, "dg_m_grouped_layout_masked", MASKED, status, needle, **change)


SCATTER = dict(x=P, w=None, row=P, slot=P, a=P, sfa=P, T=4, k=2, M=128, K=256, pow2=0, stream=None)
MSCATTER = dict(x=P, w=None, row=P, slot=P, a=P, sfa=P, T=4, k=2, G=4, m=16, K=256, pow2=0, stream=None)
KSCATTER = dict(x=P, w=None, slot=P, a=P, sfa=P, T=4, k=2, K=256, N=64, pow2=0, stream=None)
POINTERS = [
    (dict(x=None), INVALID, "NULL"), (dict(slot=None), INVALID, "NULL"), (dict(a=None), INVALID, "NULL"),
    (dict(sfa=None), INVALID, "NULL"), (dict(x=BY8), INVALID, "16-byte"), (dict(a=BY8), INVALID, "16-byte"),
    (dict(sfa=BY2), INVALID, "4-byte"), (dict(w=BY2), INVALID, "4-byte"), (dict(slot=ODD), INVALID, "4-byte"),
    (dict(T=-3), INVALID, "T=-3"), (dict(k=0), INVALID, "top_k"), (dict(T=2**30, k=4), UNSUPPORTED, "choices"),
    (dict(K=200), INVALID, "multiple of 128"), (dict(K=-128), INVALID, "negative"),
]


@pytest.mark.parametrize("fn,base", [("dg_m_grouped_scatter_fp8_contiguous", SCATTER),
                                     ("dg_m_grouped_scatter_fp8_masked", MSCATTER),
                                     ("dg_k_grouped_scatter_fp8", KSCATTER)])
@pytest.mark.parametrize("change,status,needle", POINTERS, ids=str)
def test_scatters(lib, fn, base, change, status, needle):
    refused(lib, fn, base, status, needle, **change)


def test_scatters_own_rules(lib):
    refused(lib, "dg_m_grouped_scatter_fp8_contiguous", SCATTER, INVALID, "NULL", row=None)
    refused(lib, "dg_m_grouped_scatter_fp8_contiguous", SCATTER, INVALID, "M=-1", M=-1)
    refused(lib, "dg_m_grouped_scatter_fp8_masked", MSCATTER, INVALID, "num_groups", G=0)
    refused(lib, "dg_m_grouped_scatter_fp8_masked", MSCATTER, INVALID, "max_m", m=-1)
    refused(lib, "dg_m_grouped_scatter_fp8_masked", MSCATTER, UNSUPPORTED, "rows", G=2**16, m=2**16)
    refused(lib, "dg_k_grouped_scatter_fp8", KSCATTER, UNSUPPORTED, "multiple of 16", N=72)
    refused(lib, "dg_k_grouped_scatter_fp8", KSCATTER, INVALID, "negative", N=-16)
    for fn, base in (("dg_m_grouped_scatter_fp8_contiguous", SCATTER), ("dg_m_grouped_scatter_fp8_masked", MSCATTER)):
        refused(lib, fn, base, OK, "", T=0, x=None, row=None, a=None)
        refused(lib, fn, base, OK, "", K=0, x=None, sfa=None)
    refused(lib, "dg_k_grouped_scatter_fp8", KSCATTER, OK, "", K=0, x=None, slot=None, a=None, sfa=None)


GATHER = dict(rows=P, row=P, w=None, c=None, d=P, T=4, k=2, M=128, N=65, stream=None)
GWGRAD = dict(rows=P, row=P, g=P, gw=P, T=4, k=2, M=128, N=65, stream=None)


@pytest.mark.parametrize("fn,base", [("dg_m_grouped_gather", GATHER), ("dg_m_grouped_gather_weight_grad", GWGRAD)])
@pytest.mark.parametrize("change,status,needle", [
    (dict(rows=None), INVALID, "rows"), (dict(row=None), INVALID, "row_of"), (dict(rows=ODD), INVALID, "2-byte"),
    (dict(row=BY2), INVALID, "4-byte"), (dict(T=-1), INVALID, "T=-1"), (dict(M=-1), INVALID, "negative"),
    (dict(N=-1), INVALID, "negative"), (dict(k=65), UNSUPPORTED, "top_k"), (dict(T=2**28, k=8), UNSUPPORTED, "choices"),
], ids=str)
def test_gathers(lib, fn, base, change, status, needle):
    refused(lib, fn, base, status, needle, **change)


def test_gathers_own_rules(lib):
    refused(lib, "dg_m_grouped_gather", GATHER, INVALID, "d must", d=None)
    refused(lib, "dg_m_grouped_gather", GATHER, INVALID, "2-byte", c=ODD)
    refused(lib, "dg_m_grouped_gather", GATHER, INVALID, "4-byte", w=BY2)
    refused(lib, "dg_m_grouped_gather", GATHER, OK, "", T=0, rows=None, row=None, d=None)
    refused(lib, "dg_m_grouped_gather", GATHER, OK, "", N=0, d=None)
    refused(lib, "dg_m_grouped_gather_weight_grad", GWGRAD, INVALID, "grad_d", g=None)
    refused(lib, "dg_m_grouped_gather_weight_grad", GWGRAD, INVALID, "grad_weights", gw=None)
    refused(lib, "dg_m_grouped_gather_weight_grad", GWGRAD, OK, "", T=0, row=None, g=None, gw=None)


LORA = dict(x=P, ldx=256, a=P, b=P, scales=None, ids=P, c=None, ldc=65, d=P, ldd=65, T=4, N=65, K=256, R=16, L=3,
            stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(x=None), INVALID, "NULL"), (dict(a=None), INVALID, "NULL"), (dict(b=None), INVALID, "NULL"),
    (dict(ids=None), INVALID, "NULL"), (dict(d=None), INVALID, "NULL"), (dict(x=BY8), INVALID, "16-byte"),
    (dict(a=BY8), INVALID, "16-byte"), (dict(b=BY2), INVALID, "16-byte"), (dict(d=ODD), INVALID, "2-byte"),
    (dict(c=ODD), INVALID, "2-byte"), (dict(scales=BY2), INVALID, "4-byte"), (dict(ids=BY2), INVALID, "4-byte"),
    (dict(T=-1), INVALID, "negative"), (dict(N=-1), INVALID, "negative"), (dict(L=-1), INVALID, "num_adapters"),
    (dict(K=200), INVALID, "multiple of 128"), (dict(R=12), INVALID, "multiple of 8"), (dict(R=264), UNSUPPORTED, "R="),
    (dict(L=1025), UNSUPPORTED, "num_adapters"), (dict(ldx=255), INVALID, "ldx"), (dict(ldx=260), INVALID, "ldx"),
    (dict(ldd=64), INVALID, "ldd"), (dict(c=P, ldc=64), INVALID, "ldc"), (dict(c=P, ldc=66), INVALID, "may equal d"),
    (dict(T=0, x=None, ids=None, d=None), OK, ""), (dict(N=0, b=None, d=None), OK, ""),
], ids=str)
def test_lora(lib, change, status, needle):
    refused(lib, "dg_lora_bf16_nt", LORA, status, needle, **change)


def test_rows_bound(lib):
    assert dg.dg_m_grouped_rows_bound(0, 8) == 0
    assert dg.dg_m_grouped_rows_bound(1, 8) == 128
    assert dg.dg_m_grouped_rows_bound(8192, 8) == 8192 + 7 * 128
    for c, g in ((-1, 8), (8, -1), (2**31, 8), (2**31 - 1, 1024)):
        with pytest.raises(ValueError, match="no row bound"):
            dg.dg_m_grouped_rows_bound(c, g)


def test_rows_bound_is_never_exceeded_and_is_reached():
    rng = np.random.default_rng(0)
    for _ in range(300):
        n, g = int(rng.integers(0, 2000)), int(rng.integers(1, 20))
        bound = dg.dg_m_grouped_rows_bound(n, g)
        counts = rng.multinomial(n, rng.dirichlet(np.ones(g) * 0.3))
        assert ((counts + 127) // 128 * 128).sum() <= bound
        ones = np.bincount(np.arange(min(n, g - 1)), minlength=g)     # one choice each, the rest to the last expert
        ones[g - 1] = n - ones[:g - 1].sum()
        assert bound - ((ones + 127) // 128 * 128).sum() < 128 * 2


def test_binding_refusals():
    i32, f32, b16 = torch.int32, torch.float32, torch.bfloat16
    z = torch.zeros
    ids, w = z(4, 2, dtype=i32), z(4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        dg.dg_route_topk(z(4, 8), None, ids, w)
    with pytest.raises(ValueError, match="^topk_weights has shape"):
        dg.dg_route_topk(z(4, 8), None, ids, z(4, 3))
    with pytest.raises(TypeError, match="^logits has dtype"):
        dg.dg_route_topk(z(4, 8, dtype=torch.float16), None, ids, w)
    with pytest.raises(ValueError, match="^logits must be contiguous"):
        dg.dg_route_topk(z(8, 4).t(), None, ids, w)
    with pytest.raises(ValueError, match="score is 'tanh'"):
        dg.dg_route_topk(z(4, 8), None, ids, w, score="tanh")
    with pytest.raises(ValueError, match="^bias has shape"):
        dg.dg_route_topk(z(4, 8), z(7), ids, w)
    with pytest.raises(TypeError, match="^grad_logits has dtype"):
        dg.dg_route_topk_backward(z(4, 8), ids, w, z(4, 8, dtype=b16))
    with pytest.raises(ValueError, match="^row_of has shape"):
        dg.dg_m_grouped_layout_contiguous(ids, 0, z(128, dtype=i32), z(4, 3, dtype=i32), z(128, dtype=i32), z(8, dtype=i32))
    with pytest.raises(ValueError, match="^slot_of has shape"):
        dg.dg_m_grouped_layout_contiguous(ids, 0, z(128, dtype=i32), ids, z(127, dtype=i32), z(8, dtype=i32))
    with pytest.raises(ValueError, match="^masked_m has shape"):
        dg.dg_m_grouped_layout_masked(ids, 0, z(7, dtype=i32), ids, z(8, 5, dtype=i32))
    x = z(4, 256, dtype=b16)
    slot, a = z(128, dtype=i32), z(128, 256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="^sfa has shape"):
        dg.dg_m_grouped_scatter_fp8_contiguous(x, None, ids, slot, a, z(128, 2))
    with pytest.raises(TypeError, match="^x has dtype"):
        dg.dg_m_grouped_scatter_fp8_contiguous(x.float(), None, ids, slot, a, z(2, 128))
    with pytest.raises(ValueError, match="^weights has shape"):
        dg.dg_m_grouped_scatter_fp8_masked(x, z(4), ids, z(2, 64, dtype=i32), a.view(2, 64, 256), z(2, 2, 64))
    with pytest.raises(ValueError, match="^sfa has shape"):
        dg.dg_k_grouped_scatter_fp8(x, None, slot, 2, a, z(2, 256))
    with pytest.raises(ValueError, match="^rows has shape"):
        dg.dg_m_grouped_gather(z(5, dtype=b16), ids, None, None, x)
    with pytest.raises(ValueError, match="^d has shape"):
        dg.dg_m_grouped_gather(z(9, 255, dtype=b16), ids, None, None, x)
    with pytest.raises(ValueError, match="^grad_weights has shape"):
        dg.dg_m_grouped_gather_weight_grad(z(9, 256, dtype=b16), ids, x, z(4, 3))
    la, lb, aid, d = z(3, 16, 256, dtype=b16), z(3, 65, 16, dtype=b16), z(4, dtype=i32), z(4, 65, dtype=b16)
    with pytest.raises(ValueError, match="device tensor"):
        dg.dg_lora_bf16_nt(x, la, lb, None, aid, None, d)
    with pytest.raises(ValueError, match="^b has shape"):
        dg.dg_lora_bf16_nt(x, la, z(3, 16, 65, dtype=b16), None, aid, None, d)
    with pytest.raises(ValueError, match="^d must have contiguous rows"):
        dg.dg_lora_bf16_nt(x, la, lb, None, aid, None, z(65, 4, dtype=b16).t())
    with pytest.raises(ValueError, match="^x must have contiguous rows that do not overlap"):
        dg.dg_lora_bf16_nt(z(600, dtype=b16).as_strided((4, 256), (8, 1)), la, lb, None, aid, None, d)
    with pytest.raises(TypeError, match="^c has dtype"):
        dg.dg_lora_bf16_nt(x, la, lb, None, aid, d.float(), d)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        dg.dg_lora_bf16_nt(x, la, lb, None, aid, None, None)
