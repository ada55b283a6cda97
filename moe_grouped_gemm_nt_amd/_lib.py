"""ctypes binding of libdg.so (the C ABI in include/dg.h).

Argument marshalling only: torch tensors in, device pointers and the current
HIP stream out.  Every step of the computation runs in the library's kernels;
there is no fallback path.  A missing library raises at first use."""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libdg.so")

DG_OK = 0
DG_ERR_INVALID_ARG = -1
DG_ERR_UNSUPPORTED = -2
DG_ERR_HIP = -3

EXPORTED = [
    "dg_fp8_gemm_nt",
    "dg_fp8_gemm_nt_noalloc",
    "dg_fp8_gemm_nn",
    "dg_fp8_gemm_tn",
    "dg_fp8_gemm_tt",
    "dg_fp8_fp4_gemm_nt",
    "dg_m_grouped_fp8_gemm_nt_contiguous",
    "dg_m_grouped_fp8_gemm_nt_masked",
    "dg_m_grouped_fp8_fp4_gemm_nt_contiguous",
    "dg_m_grouped_fp8_fp4_gemm_nt_masked",
    "dg_k_grouped_fp8_gemm_tn_contiguous",
    "dg_route_topk",
    "dg_route_topk_backward",
    "dg_m_grouped_rows_bound",
    "dg_m_grouped_layout_contiguous",
    "dg_m_grouped_layout_masked",
    "dg_m_grouped_scatter_fp8_contiguous",
    "dg_m_grouped_scatter_fp8_masked",
    "dg_k_grouped_scatter_fp8",
    "dg_m_grouped_gather",
    "dg_m_grouped_gather_weight_grad",
    "dg_lora_bf16_nt",
    "dg_choose_config",
    "dg_check_grouped_layout",
    "dg_bind_stream_workspace",
    "dg_init",
    "dg_last_error",
    "dg_version",
]

_lock = threading.Lock()
_lib = None


class DGError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libdg.so once; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m moe_grouped_gemm_nt_amd.build`")
        lib = ctypes.CDLL(path)
        vp, fp, i32p, ci = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        for name in ("dg_fp8_gemm_nt", "dg_fp8_gemm_nt_noalloc", "dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt"):
            getattr(lib, name).argtypes = [vp, fp, vp, fp, vp, vp, ci, ci, ci, vp]
            getattr(lib, name).restype = ci
        lib.dg_fp8_fp4_gemm_nt.argtypes = [vp, fp, vp, vp, vp, vp, ci, ci, ci, vp]
        lib.dg_fp8_fp4_gemm_nt.restype = ci
        lib.dg_m_grouped_fp8_gemm_nt_contiguous.argtypes = [vp, fp, vp, fp, vp, vp, ci, ci, ci, ci, i32p, vp]
        lib.dg_m_grouped_fp8_gemm_nt_contiguous.restype = ci
        lib.dg_m_grouped_fp8_gemm_nt_masked.argtypes = [vp, fp, vp, fp, vp, vp, ci, ci, ci, ci, i32p, ci, vp]
        lib.dg_m_grouped_fp8_gemm_nt_masked.restype = ci
        lib.dg_m_grouped_fp8_fp4_gemm_nt_contiguous.argtypes = [vp, fp, vp, vp, vp, vp, ci, ci, ci, ci, i32p, vp]
        lib.dg_m_grouped_fp8_fp4_gemm_nt_contiguous.restype = ci
        lib.dg_m_grouped_fp8_fp4_gemm_nt_masked.argtypes = [vp, fp, vp, vp, vp, vp, ci, ci, ci, ci, i32p, ci, vp]
        lib.dg_m_grouped_fp8_fp4_gemm_nt_masked.restype = ci
        lib.dg_k_grouped_fp8_gemm_tn_contiguous.argtypes = [vp, fp, vp, fp, vp, vp, ci, ci, ci, vp, vp]
        lib.dg_k_grouped_fp8_gemm_tn_contiguous.restype = ci
        cf = ctypes.c_float
        for name, types in {
            "dg_route_topk": [vp, ci, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, ci, cf, vp],
            "dg_route_topk_backward": [vp, ci, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp],
            "dg_m_grouped_rows_bound": [ctypes.c_longlong, ci],
            "dg_m_grouped_layout_contiguous": [vp, ci, ci, ci, ci, ci, vp, vp, vp, vp, vp],
            "dg_m_grouped_layout_masked": [vp, ci, ci, ci, ci, ci, vp, vp, vp, vp],
            "dg_m_grouped_scatter_fp8_contiguous": [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, vp],
            "dg_m_grouped_scatter_fp8_masked": [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp],
            "dg_k_grouped_scatter_fp8": [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, vp],
            "dg_m_grouped_gather": [vp, vp, vp, vp, vp, ci, ci, ci, ci, vp],
            "dg_m_grouped_gather_weight_grad": [vp, vp, vp, vp, ci, ci, ci, ci, vp],
            "dg_lora_bf16_nt": [vp, ci, vp, vp, vp, vp, vp, ci, vp, ci, ci, ci, ci, ci, ci, vp],
        }.items():
            getattr(lib, name).argtypes = types
            getattr(lib, name).restype = ci
        lib.dg_choose_config.argtypes = [ci, ci, ci, ci, ci, ci, ci, ci, ctypes.POINTER(ci), ctypes.POINTER(ci)]
        lib.dg_choose_config.restype = ci
        lib.dg_bind_stream_workspace.argtypes = [vp, vp, ctypes.c_size_t]
        lib.dg_bind_stream_workspace.restype = ci
        lib.dg_check_grouped_layout.argtypes = [vp, ci, ci]
        lib.dg_check_grouped_layout.restype = ci
        lib.dg_init.argtypes = []
        lib.dg_init.restype = ci
        lib.dg_last_error.argtypes = []
        lib.dg_last_error.restype = ctypes.c_char_p
        lib.dg_version.argtypes = []
        lib.dg_version.restype = ci
        _lib = lib
        return lib


def _check(fn: str, status: int):
    if status != DG_OK:
        raise DGError(fn, status, (load().dg_last_error() or b"").decode())


_CODE_DTYPES = (torch.uint8, torch.float8_e4m3fn)
_BF16_DTYPES = (torch.bfloat16, torch.int16, torch.uint16)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U8 = (torch.uint8,)


def _ptr(t, name, dtypes, shape, allow_none=False):
    """The address of t after checking its dtype, shape and layout: the
    library sees pointers and sizes only, so a tensor of another
    shape would be read or written out of bounds by the kernels.  shape None
    skips the shape check (scales when K is not a multiple of 128, which the
    library rejects itself)."""
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} must not be None")
    if type(t) is torch.Tensor and t.dtype in dtypes and (shape is None or t.shape == shape) and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on_device(**tensors):
    """Every tensor must live on the current device: the library runs the
    call there (checked after all shapes, so shape errors name the tensor
    even for host tensors)."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a device tensor")
        if t.device.index is not None and t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}; the call runs on the current device "
                             f"cuda:{torch.cuda.current_device()}")


def _kb(K):
    """K blocks of 128, or None when K is not a multiple of 128 (rejected by the library)."""
    return K // 128 if K % 128 == 0 else None


def _sh(*dims):
    """A shape, or None when one of its sizes is unknown."""
    return None if any(x is None for x in dims) else dims


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def dg_init() -> None:
    _check("dg_init", load().dg_init())


FORMS = {"dense": 0, "contiguous": 1, "masked": 2}
AB_LAYOUTS = {"nt": 0, "tt": 1, "nn": 2, "tn": 3, "fp4": 4}


def dg_choose_config(form, rows, N, K, num_groups=1, num_cus=256, ab_layout="nt", has_c=False):
    """(configuration id, decode K splits) the calls would choose; host-only,
    touches no device.  rows is M, or expected_m for the masked form."""
    cfg, splits = ctypes.c_int(-1), ctypes.c_int(0)
    _check("dg_choose_config", load().dg_choose_config(
        FORMS[form], int(rows), int(N), int(K), int(num_groups), int(num_cus), AB_LAYOUTS[ab_layout],
        1 if has_c else 0, ctypes.byref(cfg), ctypes.byref(splits)))
    return cfg.value, splits.value


def dg_bind_stream_workspace(stream, workspace) -> None:
    """Binds a device tensor (256-byte aligned, at least 256 bytes) as the
    workspace of every later call on `stream`; workspace None removes the binding."""
    if workspace is None:
        ptr, nbytes = None, 0
    else:
        _on_device(workspace=workspace)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ptr, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check("dg_bind_stream_workspace", load().dg_bind_stream_workspace(_stream(stream), ptr, nbytes))


def dg_check_grouped_layout(grouped_layout, num_groups) -> None:
    """Host-side check of a contiguous layout (a host int32 array or tensor) against
    the one-expert-per-128-row-block contract; raises DGError naming the first
    offending block."""
    import numpy as np
    h = np.ascontiguousarray(np.asarray(grouped_layout.cpu() if isinstance(grouped_layout, torch.Tensor)
                                        else grouped_layout, dtype=np.int32))
    _check("dg_check_grouped_layout", load().dg_check_grouped_layout(
        h.ctypes.data_as(ctypes.c_void_p), int(h.size), int(num_groups)))


def dg_version() -> int:
    return load().dg_version()


def _dense(fn, a, sfa, b, sfb, c, d, M, N, K, a_shape, b_shape, stream):
    """The dense calls (every operand storage): scales sfa [K/128][M] and
    sfb [ceil(N/128)][K/128], c and d [M][N]."""
    kb, nb = _kb(K), (N + 127) // 128
    args = (_ptr(a, "a", _CODE_DTYPES, a_shape), _ptr(sfa, "sfa", _F32, _sh(kb, M)),
            _ptr(b, "b", _CODE_DTYPES, b_shape), _ptr(sfb, "sfb", _F32, _sh(nb, kb)),
            _ptr(c, "c", _BF16_DTYPES, (M, N), True), _ptr(d, "d", _BF16_DTYPES, (M, N)),
            M, N, K)
    _on_device(a=a, sfa=sfa, b=b, sfb=sfb, c=c, d=d)
    _check(fn, getattr(load(), fn)(*args, _stream(stream)))


def dg_fp8_gemm_nt(a, sfa, b, sfb, c, d, stream=None) -> None:
    """d[M][N] = bf16(c + a[M][K] . b[N][K]^T) with sfa [K/128][M], sfb [ceil(N/128)][K/128]."""
    M, K = a.shape
    N = b.shape[0]
    _dense("dg_fp8_gemm_nt", a, sfa, b, sfb, c, d, M, N, K, (M, K), (N, K), stream)


def dg_fp8_gemm_nt_noalloc(a, sfa, b, sfb, c, d, stream=None) -> None:
    """As dg_fp8_gemm_nt, with the kernels' scratch in the library's fixed
    per-device array: the call allocates no device memory."""
    M, K = a.shape
    N = b.shape[0]
    _dense("dg_fp8_gemm_nt_noalloc", a, sfa, b, sfb, c, d, M, N, K, (M, K), (N, K), stream)


def dg_fp8_gemm_nn(a, sfa, b, sfb, c, d, stream=None) -> None:
    """d[M][N] = bf16(c + a[M][K] . b[K][N]) (B stored K-major), scales as in the NT call."""
    M, K = a.shape
    N = b.shape[1]
    _dense("dg_fp8_gemm_nn", a, sfa, b, sfb, c, d, M, N, K, (M, K), (K, N), stream)


def dg_fp8_gemm_tn(a, sfa, b, sfb, c, d, stream=None) -> None:
    """d[M][N] = bf16(c + a[K][M]^T . b[K][N]) (both operands stored K-major)."""
    K, M = a.shape
    N = b.shape[1]
    _dense("dg_fp8_gemm_tn", a, sfa, b, sfb, c, d, M, N, K, (K, M), (K, N), stream)


def dg_fp8_gemm_tt(a, sfa, b, sfb, c, d, stream=None) -> None:
    """d[M][N] = bf16(c + a[K][M]^T . b[N][K]^T) (A stored K-major)."""
    K, M = a.shape
    N = b.shape[0]
    _dense("dg_fp8_gemm_tt", a, sfa, b, sfb, c, d, M, N, K, (K, M), (N, K), stream)


def dg_fp8_fp4_gemm_nt(a, sfa, b, sfb, c, d, stream=None) -> None:
    """d[M][N] = bf16(c + a[M][K] . dequant(b)^T): b packed E2M1 [N][K/2], sfb int32 [K/128][N]
    (four E8M0 exponents per int, one per 32 K values)."""
    M, K = a.shape
    N = b.shape[0]
    kb = _kb(K)
    args = (_ptr(a, "a", _CODE_DTYPES, (M, K)), _ptr(sfa, "sfa", _F32, _sh(kb, M)),
            _ptr(b, "b", _U8, (N, K // 2)), _ptr(sfb, "sfb", _I32, _sh(kb, N)),
            _ptr(c, "c", _BF16_DTYPES, (M, N), True), _ptr(d, "d", _BF16_DTYPES, (M, N)),
            M, N, K)
    _on_device(a=a, sfa=sfa, b=b, sfb=sfb, c=c, d=d)
    _check("dg_fp8_fp4_gemm_nt", load().dg_fp8_fp4_gemm_nt(*args, _stream(stream)))


def dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, c, d, grouped_layout, stream=None) -> None:
    """Contiguous M-grouped form: a [M][K], b [G][N][K], sfa [K/128][M],
    sfb [G][ceil(N/128)][K/128], grouped_layout int32 [M]."""
    M, K = a.shape
    G, N, _ = b.shape
    kb = _kb(K)
    args = (_ptr(a, "a", _CODE_DTYPES, (M, K)), _ptr(sfa, "sfa", _F32, _sh(kb, M)),
            _ptr(b, "b", _CODE_DTYPES, (G, N, K)), _ptr(sfb, "sfb", _F32, _sh(G, (N + 127) // 128, kb)),
            _ptr(c, "c", _BF16_DTYPES, (M, N), True), _ptr(d, "d", _BF16_DTYPES, (M, N)), M, N, K, G,
            _ptr(grouped_layout, "grouped_layout", _I32, (M,)))
    _on_device(a=a, sfa=sfa, b=b, sfb=sfb, c=c, d=d, grouped_layout=grouped_layout)
    _check("dg_m_grouped_fp8_gemm_nt_contiguous", load().dg_m_grouped_fp8_gemm_nt_contiguous(*args, _stream(stream)))


def dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, c, d, masked_m, expected_m, stream=None) -> None:
    """Masked M-grouped form: a [G][max_m][K], b [G][N][K], sfa [G][K/128][max_m],
    sfb [G][ceil(N/128)][K/128], masked_m int32 [G] on the device."""
    G, max_m, K = a.shape
    N = b.shape[1]
    kb = _kb(K)
    args = (_ptr(a, "a", _CODE_DTYPES, (G, max_m, K)), _ptr(sfa, "sfa", _F32, _sh(G, kb, max_m)),
            _ptr(b, "b", _CODE_DTYPES, (G, N, K)), _ptr(sfb, "sfb", _F32, _sh(G, (N + 127) // 128, kb)),
            _ptr(c, "c", _BF16_DTYPES, (G, max_m, N), True), _ptr(d, "d", _BF16_DTYPES, (G, max_m, N)),
            max_m, N, K, G, _ptr(masked_m, "masked_m", _I32, (G,)), int(expected_m))
    _on_device(a=a, sfa=sfa, b=b, sfb=sfb, c=c, d=d, masked_m=masked_m)
    _check("dg_m_grouped_fp8_gemm_nt_masked", load().dg_m_grouped_fp8_gemm_nt_masked(*args, _stream(stream)))


def dg_k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, c, d, ks, stream=None) -> None:
    """K-grouped TN form: a [K][M], b [K][N], sfa [K/128][M], sfb [K/128][N], c and d fp32
    [G][M][N]; ks is a host sequence of per-group K sizes (multiples of 128) summing to K."""
    K, M = a.shape
    N = b.shape[1]
    ks = [int(k) for k in ks]
    # sizes that are negative or not multiples of 128 are the library's to reject
    if all(k >= 0 and k % 128 == 0 for k in ks) and sum(ks) != K:
        raise ValueError(f"the group sizes sum to {sum(ks)}; a has K = {K} rows")
    G = len(ks)
    kb = _kb(K)
    ks_host = (ctypes.c_int32 * G)(*ks)
    args = (_ptr(a, "a", _CODE_DTYPES, (K, M)), _ptr(sfa, "sfa", _F32, _sh(kb, M)),
            _ptr(b, "b", _CODE_DTYPES, (K, N)), _ptr(sfb, "sfb", _F32, _sh(kb, N)),
            _ptr(c, "c", _F32, (G, M, N), True), _ptr(d, "d", _F32, (G, M, N)), M, N, G,
            ctypes.cast(ks_host, ctypes.c_void_p))
    _on_device(a=a, sfa=sfa, b=b, sfb=sfb, c=c, d=d)
    _check("dg_k_grouped_fp8_gemm_tn_contiguous", load().dg_k_grouped_fp8_gemm_tn_contiguous(*args, _stream(stream)))


def dg_m_grouped_fp8_fp4_gemm_nt_contiguous(a, sfa, b, sfb, c, d, grouped_layout, stream=None) -> None:
    """Contiguous M-grouped FP8 x FP4 form: a [M][K], b packed [G][N][K/2], sfb int32 [G][K/128][N]."""
    M, K = a.shape
    G, N, _ = b.shape
    kb = _kb(K)
    args = (_ptr(a, "a", _CODE_DTYPES, (M, K)), _ptr(sfa, "sfa", _F32, _sh(kb, M)),
            _ptr(b, "b", _U8, (G, N, K // 2)), _ptr(sfb, "sfb", _I32, _sh(G, kb, N)),
            _ptr(c, "c", _BF16_DTYPES, (M, N), True), _ptr(d, "d", _BF16_DTYPES, (M, N)), M, N, K, G,
            _ptr(grouped_layout, "grouped_layout", _I32, (M,)))
    _on_device(a=a, sfa=sfa, b=b, sfb=sfb, c=c, d=d, grouped_layout=grouped_layout)
    _check("dg_m_grouped_fp8_fp4_gemm_nt_contiguous", load().dg_m_grouped_fp8_fp4_gemm_nt_contiguous(*args, _stream(stream)))


def dg_m_grouped_fp8_fp4_gemm_nt_masked(a, sfa, b, sfb, c, d, masked_m, expected_m, stream=None) -> None:
    """Masked M-grouped FP8 x FP4 form: a [G][max_m][K], b packed [G][N][K/2], sfb int32 [G][K/128][N]."""
    G, max_m, K = a.shape
    N = b.shape[1]
    kb = _kb(K)
    args = (_ptr(a, "a", _CODE_DTYPES, (G, max_m, K)), _ptr(sfa, "sfa", _F32, _sh(G, kb, max_m)),
            _ptr(b, "b", _U8, (G, N, K // 2)), _ptr(sfb, "sfb", _I32, _sh(G, kb, N)),
            _ptr(c, "c", _BF16_DTYPES, (G, max_m, N), True), _ptr(d, "d", _BF16_DTYPES, (G, max_m, N)),
            max_m, N, K, G, _ptr(masked_m, "masked_m", _I32, (G,)), int(expected_m))
    _on_device(a=a, sfa=sfa, b=b, sfb=sfb, c=c, d=d, masked_m=masked_m)
    _check("dg_m_grouped_fp8_fp4_gemm_nt_masked", load().dg_m_grouped_fp8_fp4_gemm_nt_masked(*args, _stream(stream)))


# ---- the operators around the products -------------------------------------
_LOGITS = (torch.float32, torch.bfloat16)
_BF16 = (torch.bfloat16,)
SCORES = {"softmax": 0, "sigmoid": 1}


def _run(fn, tensors, args, stream):
    """Checks that every tensor (None left out) lives on the current device, then makes the call.
    These calls take a few microseconds on the device, so the host side is kept as short."""
    here = torch.cuda.current_device() if torch.cuda.is_initialized() else None
    for t in tensors.values():
        if t is not None and t.get_device() != here:
            _on_device(**tensors)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(here)
    else:
        stream = _stream(stream)
    status = getattr(_lib or load(), fn)(*args, stream)
    if status:
        _check(fn, status)


def _score(score):
    if score not in SCORES:
        raise ValueError(f"score is {score!r}; expected one of {sorted(SCORES)}")
    return SCORES[score]


def _rank(t, name, dims):
    """Whether t is a tensor of that many dimensions: sizes are read from it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() not in dims:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {' or '.join(map(str, dims))} dimensions")
    return t.shape


def dg_route_topk(logits, bias, topk_ids, topk_weights, score="softmax", num_groups=1, topk_groups=1, group_top=1,
                  renormalize=True, scale=1.0, stream=None) -> None:
    """Chooses each token's experts: topk_ids int32 and topk_weights fp32 [T][top_k] from logits [T][E]
    (fp32 or bf16) and an optional fp32 bias [E] that steers the choice only."""
    T, E = _rank(logits, "logits", (2,))
    k = _rank(topk_ids, "topk_ids", (2,))[1]
    args = (_ptr(logits, "logits", _LOGITS, None), 0 if logits.dtype == torch.float32 else 1,
            _ptr(bias, "bias", _F32, (E,), True), _ptr(topk_ids, "topk_ids", _I32, (T, k)),
            _ptr(topk_weights, "topk_weights", _F32, (T, k)), T, E, k, _score(score), int(num_groups),
            int(topk_groups), int(group_top), 1 if renormalize else 0, float(scale))
    _run("dg_route_topk", dict(logits=logits, bias=bias, topk_ids=topk_ids, topk_weights=topk_weights), args, stream)


def dg_route_topk_backward(logits, topk_ids, grad_weights, grad_logits, score="softmax", renormalize=True, scale=1.0,
                           stream=None) -> None:
    """grad_logits [T][E] (of the logits' type) from the gradient of the forward call's weights [T][top_k]."""
    T, E = _rank(logits, "logits", (2,))
    k = _rank(topk_ids, "topk_ids", (2,))[1]
    args = (_ptr(logits, "logits", _LOGITS, None), 0 if logits.dtype == torch.float32 else 1,
            _ptr(topk_ids, "topk_ids", _I32, (T, k)), _ptr(grad_weights, "grad_weights", _F32, (T, k)),
            _ptr(grad_logits, "grad_logits", (logits.dtype,), (T, E)), T, E, k, _score(score),
            1 if renormalize else 0, float(scale))
    _run("dg_route_topk_backward", dict(logits=logits, topk_ids=topk_ids, grad_weights=grad_weights,
                                        grad_logits=grad_logits), args, stream)


def dg_m_grouped_rows_bound(choices, num_groups) -> int:
    """The most rows the contiguous layout of `choices` choices over num_groups experts can need."""
    rows = load().dg_m_grouped_rows_bound(int(choices), int(num_groups))
    if rows < 0:
        raise ValueError(f"no row bound for {choices} choices over {num_groups} groups")
    return rows


def dg_m_grouped_layout_contiguous(topk_ids, first_expert, grouped_layout, row_of, slot_of, counts,
                                   stream=None) -> None:
    """Rows for the contiguous products from topk_ids int32 [T][top_k]: grouped_layout and slot_of int32 [M],
    row_of int32 [T][top_k], counts int32 [num_groups]."""
    T, k = _rank(topk_ids, "topk_ids", (2,))
    M, G = _rank(grouped_layout, "grouped_layout", (1,))[0], _rank(counts, "counts", (1,))[0]
    args = (_ptr(topk_ids, "topk_ids", _I32, None), T, k, int(first_expert), G, M,
            _ptr(grouped_layout, "grouped_layout", _I32, None), _ptr(row_of, "row_of", _I32, (T, k)),
            _ptr(slot_of, "slot_of", _I32, (M,)), _ptr(counts, "counts", _I32, None))
    _run("dg_m_grouped_layout_contiguous", dict(topk_ids=topk_ids, grouped_layout=grouped_layout, row_of=row_of,
                                                slot_of=slot_of, counts=counts), args, stream)


def dg_m_grouped_layout_masked(topk_ids, first_expert, masked_m, row_of, slot_of, stream=None) -> None:
    """Rows for the masked products: masked_m int32 [num_groups], row_of int32 [T][top_k],
    slot_of int32 [num_groups][max_m]."""
    T, k = _rank(topk_ids, "topk_ids", (2,))
    G, m = _rank(slot_of, "slot_of", (2,))
    args = (_ptr(topk_ids, "topk_ids", _I32, None), T, k, int(first_expert), G, m,
            _ptr(masked_m, "masked_m", _I32, (G,)), _ptr(row_of, "row_of", _I32, (T, k)),
            _ptr(slot_of, "slot_of", _I32, None))
    _run("dg_m_grouped_layout_masked", dict(topk_ids=topk_ids, masked_m=masked_m, row_of=row_of, slot_of=slot_of),
         args, stream)


def dg_m_grouped_scatter_fp8_contiguous(x, weights, row_of, slot_of, a, sfa, pow2_scales=False, stream=None) -> None:
    """The tokens' rows x bf16 [T][K], times weights fp32 [T][top_k] if given, quantised into
    a [M][K] (e4m3 codes) and sfa fp32 [K/128][M] at the rows row_of / slot_of."""
    T, K = _rank(x, "x", (2,))
    k = _rank(row_of, "row_of", (2,))[1]
    M = _rank(a, "a", (2,))[0]
    args = (_ptr(x, "x", _BF16, None), _ptr(weights, "weights", _F32, (T, k), True),
            _ptr(row_of, "row_of", _I32, (T, k)), _ptr(slot_of, "slot_of", _I32, (M,)),
            _ptr(a, "a", _CODE_DTYPES, (M, K)), _ptr(sfa, "sfa", _F32, _sh(_kb(K), M)), T, k, M, K,
            1 if pow2_scales else 0)
    _run("dg_m_grouped_scatter_fp8_contiguous", dict(x=x, weights=weights, row_of=row_of, slot_of=slot_of, a=a,
                                                     sfa=sfa), args, stream)


def dg_m_grouped_scatter_fp8_masked(x, weights, row_of, slot_of, a, sfa, pow2_scales=False, stream=None) -> None:
    """As the contiguous form, into a [G][max_m][K] and sfa fp32 [G][K/128][max_m]; slot_of [G][max_m]."""
    T, K = _rank(x, "x", (2,))
    k = _rank(row_of, "row_of", (2,))[1]
    G, m, _ = _rank(a, "a", (3,))
    args = (_ptr(x, "x", _BF16, None), _ptr(weights, "weights", _F32, (T, k), True),
            _ptr(row_of, "row_of", _I32, (T, k)), _ptr(slot_of, "slot_of", _I32, (G, m)),
            _ptr(a, "a", _CODE_DTYPES, (G, m, K)), _ptr(sfa, "sfa", _F32, _sh(G, _kb(K), m)), T, k, G, m, K,
            1 if pow2_scales else 0)
    _run("dg_m_grouped_scatter_fp8_masked", dict(x=x, weights=weights, row_of=row_of, slot_of=slot_of, a=a, sfa=sfa),
         args, stream)


def dg_k_grouped_scatter_fp8(x, weights, slot_of, top_k, a, sfa, pow2_scales=False, stream=None) -> None:
    """The rows x bf16 [T][N] (times weights fp32 [T][top_k]) as a K-grouped operand: a [K][N] codes,
    sfa fp32 [K/128][N], zeros in rows without a choice; slot_of int32 [K]."""
    T, N = _rank(x, "x", (2,))
    K = _rank(a, "a", (2,))[0]
    k = int(top_k)
    args = (_ptr(x, "x", _BF16, None), _ptr(weights, "weights", _F32, (T, k), True),
            _ptr(slot_of, "slot_of", _I32, (K,)), _ptr(a, "a", _CODE_DTYPES, (K, N)),
            _ptr(sfa, "sfa", _F32, _sh(_kb(K), N)), T, k, K, N, 1 if pow2_scales else 0)
    _run("dg_k_grouped_scatter_fp8", dict(x=x, weights=weights, slot_of=slot_of, a=a, sfa=sfa), args, stream)


def _rows2(rows):
    """(M, N) of the experts' rows, [M][N] or the masked form's [G][max_m][N]."""
    s = _rank(rows, "rows", (2, 3))
    return (s[0], s[1]) if len(s) == 2 else (s[0] * s[1], s[2])


def dg_m_grouped_gather(rows, row_of, weights, c, d, stream=None) -> None:
    """d[t] = bf16(c[t] + sum_j weights[t][j] * rows[row_of[t][j]]): rows bf16 [M][N] or [G][max_m][N],
    row_of int32 and weights fp32 (or None) [T][top_k], c (or None) and d bf16 [T][N]."""
    M, N = _rows2(rows)
    T, k = _rank(row_of, "row_of", (2,))
    args = (_ptr(rows, "rows", _BF16, None), _ptr(row_of, "row_of", _I32, None),
            _ptr(weights, "weights", _F32, (T, k), True), _ptr(c, "c", _BF16, (T, N), True),
            _ptr(d, "d", _BF16, (T, N)), T, k, M, N)
    _run("dg_m_grouped_gather", dict(rows=rows, row_of=row_of, weights=weights, c=c, d=d), args, stream)


def dg_m_grouped_gather_weight_grad(rows, row_of, grad_d, grad_weights, stream=None) -> None:
    """grad_weights[t][j] = grad_d[t] . rows[row_of[t][j]]: grad_d bf16 [T][N], grad_weights fp32 [T][top_k]."""
    M, N = _rows2(rows)
    T, k = _rank(row_of, "row_of", (2,))
    args = (_ptr(rows, "rows", _BF16, None), _ptr(row_of, "row_of", _I32, None),
            _ptr(grad_d, "grad_d", _BF16, (T, N)), _ptr(grad_weights, "grad_weights", _F32, (T, k)), T, k, M, N)
    _run("dg_m_grouped_gather_weight_grad", dict(rows=rows, row_of=row_of, grad_d=grad_d, grad_weights=grad_weights),
         args, stream)


def _strided(t, name, shape, allow_none=False):
    """(address, row stride) of a bf16 matrix whose rows are contiguous and may lie apart (a column slice)."""
    if t is None and allow_none:
        return None, shape[1]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _BF16:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {_BF16}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    ld = t.stride(0) if shape[0] > 1 else shape[1]
    if (shape[1] > 1 and t.stride(1) != 1) or ld < shape[1]:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    if ld >= 1 << 31:
        raise ValueError(f"{name} has rows {ld} elements apart; at most 2^31 - 1")
    return t.data_ptr(), ld


def dg_lora_bf16_nt(x, a, b, scales, adapter_ids, c, d, stream=None) -> None:
    """d[t] = bf16(c[t] + scales[i] * b[i] . (a[i] . x[t])), i = adapter_ids[t]: x bf16 [T][K],
    a bf16 [L][R][K], b bf16 [L][N][R], scales fp32 [L] or None, adapter_ids int32 [T], c (or None) and
    d bf16 [T][N].  The rows of x, c and d may lie apart."""
    T, K = _rank(x, "x", (2,))
    L, R, _ = _rank(a, "a", (3,))
    N = _rank(d, "d", (2,))[1]
    px, ldx = _strided(x, "x", (T, K))
    pc, ldc = _strided(c, "c", (T, N), True)
    pd, ldd = _strided(d, "d", (T, N))
    args = (px, ldx, _ptr(a, "a", _BF16, (L, R, K)), _ptr(b, "b", _BF16, (L, N, R)),
            _ptr(scales, "scales", _F32, (L,), True), _ptr(adapter_ids, "adapter_ids", _I32, (T,)), pc, ldc, pd, ldd,
            T, N, K, R, L)
    _run("dg_lora_bf16_nt", dict(x=x, a=a, b=b, scales=scales, adapter_ids=adapter_ids, c=c, d=d), args, stream)
