"""Sizes beyond what one launch of a kernel around the products can cover are
refused on the host, and include/dg.h names the limit.  No GPU."""
import ctypes
import os

import pytest

from moe_grouped_gemm_nt_amd import _lib

P = ctypes.c_void_p(0x100000)                  # aligned, never read: every call here ends on the host
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from moe_grouped_gemm_nt_amd import build
        build.build()
    return _lib.load()


LIMITS = [
    # entry, its arguments with one beyond the limit, what the message and the header's comment say
    ("dg_k_grouped_scatter_fp8", [P, P, P, P, P, 4, 2, 128, 2 ** 30, 0, None], "N=1073741824", "N below 2^30"),
    ("dg_lora_bf16_nt", [P, 128, P, P, P, P, None, 0, P, 2 ** 24, 4, 2 ** 24, 128, 16, 3, None], "N=16777216 exceeds 16776960",
     "N at most 16776960"),
    ("dg_m_grouped_gather", [P, P, P, P, P, 4, 2, 128, 2 ** 30 + 1, None], "N=1073741825", "N at most 2^30"),
    ("dg_m_grouped_gather_weight_grad", [P, P, P, P, 4, 2, 128, 2 ** 30 + 1, None], "N=1073741825", "N at most 2^30"),
    ("dg_m_grouped_layout_contiguous", [P, 2 ** 29 + 1, 2, 0, 8, 128, P, P, P, P, None], "choices exceed 2^30", "T * top_k at most 2^30"),
]


def section(name):
    with open(os.path.join(ROOT, "include", "dg.h")) as f:
        header = f.read()
    at = header.index("int " + name + "(")
    text = header[header.rindex("/*", 0, at):at]
    general = header[header.index("The operators around the products ---"):]
    return " ".join((general[:general.index("*/")] + text).replace("\n * ", " ").split())


@pytest.mark.parametrize("name,args,message,said", LIMITS, ids=[c[0] for c in LIMITS])
def test_limits_are_refused_and_named(lib, name, args, message, said):
    assert getattr(lib, name)(*args) == _lib.DG_ERR_UNSUPPORTED
    assert message in lib.dg_last_error().decode()
    assert said in section(name)
