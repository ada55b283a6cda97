"""What the balance loss, the 4-bit products and the gradients' calls refuse, on the
host and without a GPU: through the C ABI (before any HIP call) and through the
Python binding.  And that include/dg.h names the calls' limits and scratch."""
import ctypes
import os
import re

import pytest
import torch

import moe_grouped_gemm_nt_amd as dg
from moe_grouped_gemm_nt_amd import _lib

INVALID, UNSUPPORTED, OK = _lib.DG_ERR_INVALID_ARG, _lib.DG_ERR_UNSUPPORTED, _lib.DG_OK
P = ctypes.c_void_p(0x100000)                  # aligned, never read: every call here ends on the host
ODD, BY2, BY4, BY8 = (ctypes.c_void_p(0x100000 + n) for n in (1, 2, 4, 8))
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


BALANCE = dict(logits=P, type=0, ids=P, starts=P, loss=P, counts=P, T=4, E=64, k=8, S=3, score=1, scale=1.0, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(logits=None), INVALID, "logits must not be NULL"), (dict(ids=None), INVALID, "topk_ids"),
    (dict(loss=None), INVALID, "loss"), (dict(counts=None), INVALID, "counts"), (dict(starts=None), INVALID, "num_seqs=3"),
    (dict(type=2), INVALID, "logits_type"), (dict(score=2), INVALID, "score"), (dict(T=-1), INVALID, "negative"),
    (dict(S=-1), INVALID, "negative"), (dict(E=0), INVALID, "top_k"), (dict(k=0), INVALID, "top_k"),
    (dict(k=65), INVALID, "top_k"), (dict(E=1025), UNSUPPORTED, "experts"), (dict(E=512, k=65), UNSUPPORTED, "choices"),
    (dict(T=2 ** 28), UNSUPPORTED, "2^30"), (dict(logits=BY2), INVALID, "aligned"), (dict(starts=BY2), INVALID, "aligned"),
    (dict(counts=ODD), INVALID, "aligned"), (dict(loss=BY2), INVALID, "4-byte"), (dict(ids=BY2), INVALID, "4-byte"),
    (dict(S=0, loss=None, counts=None), OK, ""),
], ids=str)
def test_balance(lib, change, status, needle):
    refused(lib, "dg_route_balance", BALANCE, status, needle, **change)


BACK = dict(logits=P, type=1, counts=P, starts=P, gl=P, c=P, out=P, T=4, E=64, k=8, S=3, score=0, scale=1.0, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(logits=None), INVALID, "NULL"), (dict(counts=None), INVALID, "counts"), (dict(out=None), INVALID, "grad_logits"),
    (dict(starts=None), INVALID, "num_seqs"), (dict(type=-1), INVALID, "logits_type"), (dict(E=1025), UNSUPPORTED, "experts"),
    (dict(k=65), INVALID, "top_k"), (dict(c=ODD), INVALID, "aligned"), (dict(out=ODD), INVALID, "aligned"),
    (dict(gl=BY2), INVALID, "aligned"), (dict(type=0, c=BY2), INVALID, "aligned"),
    (dict(T=2 ** 28), UNSUPPORTED, "2^30"), (dict(T=0, logits=None, out=None), OK, ""),
], ids=str)
def test_balance_backward(lib, change, status, needle):
    refused(lib, "dg_route_balance_backward", BACK, status, needle, **change)


FP4 = dict(x=P, ldx=256, b=P, sfb=P, c=P, ldc=65, d=P, ldd=65, M=4, N=65, K=256, stream=None)
INT4 = dict(x=P, ldx=256, b=P, scales=P, type=1, zeros=P, group=64, c=P, ldc=65, d=P, ldd=65, M=4, N=65, K=256, stream=None)
FP4X = dict(x=P, ldx=256, rows=4, ids=P, b=P, sfb=P, c=P, ldc=65, d=P, ldd=65, T=4, k=2, first=0, G=3, N=65, K=256,
            stream=None)
INT4X = dict(x=P, ldx=256, rows=8, ids=P, b=P, scales=P, type=0, zeros=None, group=32, c=P, ldc=65, d=P, ldd=65, T=4, k=2,
             first=0, G=3, N=65, K=256, stream=None)
CALLS = [("dg_bf16_fp4_gemv_nt", FP4), ("dg_bf16_int4_gemv_nt", INT4), ("dg_m_grouped_bf16_fp4_gemv_nt_topk", FP4X),
         ("dg_m_grouped_bf16_int4_gemv_nt_topk", INT4X)]


@pytest.mark.parametrize("fn,base", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("change,status,needle", [
    (dict(x=None), INVALID, "NULL"), (dict(b=None), INVALID, "NULL"), (dict(d=None), INVALID, "d must not be NULL"),
    (dict(x=BY8), INVALID, "16-byte"), (dict(b=BY8), INVALID, "16-byte"), (dict(d=ODD), INVALID, "2-byte"),
    (dict(c=ODD), INVALID, "2-byte"), (dict(K=100), INVALID, "multiple of 128"), (dict(K=-128), INVALID, "negative"),
    (dict(N=-1), INVALID, "negative"), (dict(ldx=255), INVALID, "ldx"), (dict(ldx=260), INVALID, "ldx"),
    (dict(ldd=64), INVALID, "ldd"), (dict(ldc=64), INVALID, "ldc"), (dict(ldc=70), INVALID, "c may equal d"),
    (dict(N=2 ** 20 + 1, ldc=2 ** 21, ldd=2 ** 21), UNSUPPORTED, "N=1048577 exceeds 2^20"),
    (dict(K=2 ** 24 + 128, ldx=2 ** 25), UNSUPPORTED, "exceeds 2^24"), (dict(N=0, d=None), OK, ""),
], ids=str)
def test_products(lib, fn, base, change, status, needle):
    refused(lib, fn, base, status, needle, **change)


def test_products_own_rules(lib):
    for fn, base in CALLS[:2]:
        refused(lib, fn, base, INVALID, "M=-1", M=-1)
        refused(lib, fn, base, OK, "", M=0, x=None, d=None)
    for fn, base in CALLS[2:]:
        refused(lib, fn, base, INVALID, "T=-1", T=-1)
        refused(lib, fn, base, INVALID, "top_k=0", k=0)
        refused(lib, fn, base, UNSUPPORTED, "2^30", T=2 ** 30)
        refused(lib, fn, base, INVALID, "x_rows", rows=5)
        refused(lib, fn, base, INVALID, "num_groups", G=-1)
        refused(lib, fn, base, UNSUPPORTED, "num_groups", G=1025)
        refused(lib, fn, base, INVALID, "first_expert", first=-1)
        refused(lib, fn, base, INVALID, "topk_ids", ids=None)
        refused(lib, fn, base, INVALID, "topk_ids", ids=BY2)
        refused(lib, fn, base, OK, "", T=0, rows=0, x=None, ids=None, d=None)
    for fn, base in (CALLS[0], CALLS[2]):
        refused(lib, fn, base, INVALID, "NULL", sfb=None)
        refused(lib, fn, base, INVALID, "scales", sfb=BY2)
    for fn, base in (CALLS[1], CALLS[3]):
        refused(lib, fn, base, INVALID, "NULL", scales=None)
        refused(lib, fn, base, INVALID, "group_size", group=256)
        refused(lib, fn, base, INVALID, "group_size", group=0)
        refused(lib, fn, base, INVALID, "scales_type", type=7)
        refused(lib, fn, base, INVALID, "scales", type=0, scales=BY2)
        refused(lib, fn, base, INVALID, "scales", type=1, scales=ODD)


def arrays(pointers, types=None, sizes=None):
    n = len(pointers)
    return ((ctypes.c_void_p * n)(*pointers), (ctypes.c_int * n)(*(types or [0] * n)),
            (ctypes.c_longlong * n)(*(sizes or [16] * n)))


def test_gradients(lib):
    at = 0x100000
    p, t, s = arrays([at, at + 64])
    o, _, _ = arrays([at + 4096, at + 8192])

    def norm(status, needle, grads=p, types=t, sizes=s, n=2, out=P):
        assert lib.dg_grad_norm(grads, types, sizes, n, out, None) == status
        assert needle in lib.dg_last_error().decode()

    def clip(status, needle, grads=p, out=o, types=t, sizes=s, n=2, nrm=ctypes.c_void_p(0x200000), most=1.0):
        assert lib.dg_grad_clip(grads, out, types, sizes, n, nrm, most, None) == status
        assert needle in lib.dg_last_error().decode()

    for call in (norm, clip):
        call(INVALID, "num_tensors", n=-1)
        call(UNSUPPORTED, "2^20", n=2 ** 20 + 1)
        call(INVALID, "NULL", grads=None)
        call(INVALID, "NULL", types=None)
        call(INVALID, "NULL", sizes=None)
        call(INVALID, "types[1]=2", types=arrays([1, 1], [0, 2])[1])
        call(INVALID, "sizes[0]=-1", sizes=arrays([1, 1], None, [-1, 4])[2])
        call(UNSUPPORTED, "2^43", sizes=arrays([1, 1], None, [2 ** 43 + 1, 4])[2])
        call(INVALID, "grads[1] must not be NULL", grads=arrays([at, 0])[0])
        call(INVALID, "aligned", grads=arrays([at, at + 66])[0])
        call(INVALID, "aligned", grads=arrays([at + 1, at + 64])[0], types=arrays([1, 1], [1, 1])[1])
    norm(INVALID, "norm", out=None)
    norm(INVALID, "norm", out=BY2)
    clip(INVALID, "norm", nrm=None)
    clip(INVALID, "max_norm", most=-1.0)
    clip(INVALID, "max_norm", most=float("nan"))
    clip(INVALID, "out must not be NULL", out=None)
    clip(INVALID, "out[0] must not be NULL", out=arrays([0, at])[0])
    clip(INVALID, "out[1] must be aligned", out=arrays([at + 4096, at + 8193])[0])
    # the same memory twice, a part of another tensor, the norm's own place
    clip(INVALID, "apart", out=arrays([at + 4096, at + 4096])[0])
    clip(INVALID, "apart", out=arrays([at + 4096, at + 4096 + 60])[0])
    clip(INVALID, "apart", out=arrays([at + 4, at + 64])[0])
    clip(INVALID, "apart", out=arrays([at + 64, at])[0])
    clip(INVALID, "apart", out=arrays([at, at + 64 + 60])[0])
    clip(INVALID, "apart", grads=arrays([at, at])[0], out=arrays([at, at])[0])
    clip(INVALID, "apart", nrm=ctypes.c_void_p(at + 4096 + 60))


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


BF, I, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.mark.parametrize("call,error", [
    (lambda: dg.dg_route_balance(t(4, 8), t(4, 2, dtype=I), None, t(2), t(2, 8, dtype=I)), "seq_starts must not be None"),
    (lambda: dg.dg_route_balance(t(4, 8), t(4, 2, dtype=I), t(2, dtype=I), t(2), t(2, 8, dtype=I)), "seq_starts has shape"),
    (lambda: dg.dg_route_balance(t(4, 8), t(3, 2, dtype=I), None, t(1), t(1, 8, dtype=I)), "topk_ids has shape"),
    (lambda: dg.dg_route_balance(t(4, 8), t(4, 2, dtype=I), None, t(1), t(1, 7, dtype=I)), "counts has shape"),
    (lambda: dg.dg_route_balance(t(4, 8), t(4, 2, dtype=I), None, t(1), t(1, 8, dtype=I), score="relu"), "score"),
    (lambda: dg.dg_route_balance(t(4, 8).t(), t(8, 2, dtype=I), None, t(1), t(1, 4, dtype=I)), "contiguous"),
    (lambda: dg.dg_route_balance(t(4, 8), t(4, 2, dtype=I), None, t(1), t(1, 8, dtype=I)), "device tensor"),
    (lambda: dg.dg_route_balance_backward(t(4, 8), t(1, 8, dtype=I), None, t(2), None, t(4, 8), 2), "grad_loss has shape"),
    (lambda: dg.dg_route_balance_backward(t(4, 8), t(1, 8, dtype=I), None, None, t(4, 8, dtype=BF), t(4, 8), 2), "c has dtype"),
    (lambda: dg.dg_route_balance_backward(t(4, 8), t(1, 8, dtype=I), None, None, None, t(4, 7), 2), "grad_logits has shape"),
    (lambda: dg.dg_bf16_fp4_gemv_nt(t(2, 128, dtype=BF), t(5, 64, dtype=U8), t(1, 4, dtype=I), None, t(2, 5, dtype=BF)),
     "sfb has shape"),
    (lambda: dg.dg_bf16_fp4_gemv_nt(t(2, 128), t(5, 64, dtype=U8), t(1, 5, dtype=I), None, t(2, 5, dtype=BF)), "x has dtype"),
    (lambda: dg.dg_bf16_fp4_gemv_nt(t(2, 128, dtype=BF), t(5, 64, dtype=U8), t(1, 5, dtype=I), None, t(2, 4, dtype=BF)),
     "d has shape"),
    (lambda: dg.dg_bf16_fp4_gemv_nt(t(2, 128, dtype=BF), t(5, 63, dtype=U8), t(1, 5, dtype=I), None, t(2, 5, dtype=BF)),
     "b has shape"),
    (lambda: dg.dg_bf16_fp4_gemv_nt(t(128, 2, dtype=BF).t(), t(5, 64, dtype=U8), t(1, 5, dtype=I), None, t(2, 5, dtype=BF)),
     "contiguous rows"),
    (lambda: dg.dg_bf16_fp4_gemv_nt(t(2, 128, dtype=BF), t(5, 64, dtype=U8), t(1, 5, dtype=I), None, t(2, 5, dtype=BF)),
     "device tensor"),
    (lambda: dg.dg_bf16_int4_gemv_nt(t(2, 128, dtype=BF), t(5, 64, dtype=U8), t(3, 5), None, None, t(2, 5, dtype=BF)),
     "must divide"),
    (lambda: dg.dg_bf16_int4_gemv_nt(t(2, 128, dtype=BF), t(5, 64, dtype=U8), t(2, 5), t(1, 5, dtype=U8), None,
                                     t(2, 5, dtype=BF)), "zeros has shape"),
    (lambda: dg.dg_bf16_int4_gemv_nt(t(2, 128, dtype=BF), t(5, 64, dtype=U8), t(2, 5, dtype=torch.float16), None, None,
                                     t(2, 5, dtype=BF)), "scales has dtype"),
    (lambda: dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(t(2, 128, dtype=BF), t(2, 3, dtype=I), 0, t(4, 5, 64, dtype=U8),
                                                   t(3, 1, 5, dtype=I), None, t(6, 5, dtype=BF)), "sfb has shape"),
    (lambda: dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(t(2, 128, dtype=BF), t(2, 3, dtype=I), 0, t(4, 5, 64, dtype=U8),
                                                   t(4, 1, 5, dtype=I), None, t(5, 5, dtype=BF)), "d has shape"),
    (lambda: dg.dg_m_grouped_bf16_int4_gemv_nt_topk(t(2, 128, dtype=BF), t(2, 3, dtype=I), 0, t(4, 5, 64, dtype=U8),
                                                    t(4, 4, 6), None, None, t(6, 5, dtype=BF)), "scales has shape"),
    (lambda: dg.dg_grad_norm([t(3), t(4, dtype=torch.float16)], t(1)), "tensor 1 has dtype"),
    (lambda: dg.dg_grad_norm([t(3, 4).t()], t(1)), "contiguous"), (lambda: dg.dg_grad_norm([t(3), None], t(1)), "tensor 1"),
    (lambda: dg.dg_grad_norm([t(3)], t(2)), "norm has shape"), (lambda: dg.dg_grad_norm([t(3)], t(1)), "device tensor"),
    (lambda: dg.dg_grad_clip([t(3)], [t(4)], t(1), 1.0), "types and sizes"),
    (lambda: dg.dg_grad_clip([t(3)], [t(3, dtype=BF)], t(1), 1.0), "types and sizes"),
    (lambda: dg.dg_grad_clip([t(3)], [], t(1), 1.0), "types and sizes"),
])
def test_binding(call, error):
    with pytest.raises((ValueError, TypeError), match=re.escape(error)):
        call()


# ---- what include/dg.h says of them ---------------------------------------------
def read(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


def comment_of(name):
    header = read("include", "dg.h")
    at = re.search(rf"^int {name}\(", header, re.M).start()
    comment = header.rindex("/*", 0, at)
    return " ".join(header[comment:at].replace("\n * ", " ").split())


@pytest.mark.parametrize("name,said", [
    ("dg_route_balance", "T * top_k at most 2^30"), ("dg_route_balance", "E at most 1024"),
    ("dg_bf16_fp4_gemv_nt", "N at most 2^20"), ("dg_bf16_int4_gemv_nt", "K must be a multiple of 128 and at most 2^24"),
    ("dg_m_grouped_bf16_fp4_gemv_nt_topk", "num_groups at most 1024"), ("dg_grad_norm", "num_tensors at most 2^20"),
    ("dg_grad_norm", "at most 2^43 elements"), ("dg_grad_clip", "max_norm must not be negative"),
])
def test_limits_are_named(name, said):
    assert said in comment_of(name)


@pytest.mark.parametrize("name,uses", [
    ("dg_route_balance", True), ("dg_route_balance_backward", False), ("dg_bf16_fp4_gemv_nt", False),
    ("dg_bf16_int4_gemv_nt", False), ("dg_m_grouped_bf16_fp4_gemv_nt_topk", True),
    ("dg_m_grouped_bf16_int4_gemv_nt_topk", True), ("dg_grad_norm", True), ("dg_grad_clip", False)])
def test_the_header_names_the_calls_that_use_the_workspace(name, uses):
    assert ("Scratch: workspace" in comment_of(name)) == uses
