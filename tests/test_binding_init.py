"""The native side's table of addresses, on the CPU: init() takes all of its arguments or none, and without it no call
is made.  The addresses are those of Python functions, and the tensors are fake ones that say they are on a GPU, so that
whole calls go through.  Each case has an interpreter of its own: the table is the process's."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "moe_grouped_gemm_nt_amd")

SETUP = textwrap.dedent("""
    import ctypes, importlib.util, sys, warnings
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    warnings.simplefilter("ignore")
    spec = importlib.util.spec_from_file_location("_binding", sys.argv[1])
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    with FakeTensorMode():
        norm, logits = torch.empty(1, device="cuda"), torch.empty(2, 4, device="cuda")
        ids, counts = torch.empty(2, 1, device="cuda", dtype=torch.int32), torch.empty(1, 4, device="cuda", dtype=torch.int32)
    vp, ci = ctypes.c_void_p, ctypes.c_int
    made = []
    def function(status, *types):
        made.append(ctypes.CFUNCTYPE(ci, *types)(lambda *a: status))
        return ctypes.cast(made[-1], vp).value
    names = ["dg_route_balance", "dg_route_balance_backward", "dg_bf16_fp4_gemv_nt", "dg_bf16_int4_gemv_nt",
             "dg_m_grouped_bf16_fp4_gemv_nt_topk", "dg_m_grouped_bf16_int4_gemv_nt_topk", "dg_grad_norm", "dg_grad_clip"]
    def table(first, norm):
        at = dict.fromkeys(names, function(first, vp, ci, vp, vp, vp, vp, ci, ci, ci, ci, ci, ctypes.c_float, vp))
        at["dg_grad_norm"] = function(norm, vp, vp, vp, ci, vp, vp)
        return at
    def both():
        return (native.dg_route_balance(logits, ids, None, norm, counts, 0, 1.0, None),
                native.dg_grad_norm([], norm, None))
""")


def run(body):
    from moe_grouped_gemm_nt_amd import build
    if not os.path.exists(build.BINDING_PATH):
        build.build()
    r = subprocess.run([sys.executable, "-c", SETUP + textwrap.dedent(body), build.BINDING_PATH], capture_output=True,
                       text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "DONE" in r.stdout, (r.returncode, r.stdout[-500:], r.stderr[-1500:])


def test_calls_go_to_the_addresses():
    run("""
        native.init(table(3, 5), lambda: 0, lambda device: 77)
        assert both() == (3, 5)
        native.init(table(4, 6), lambda: 0, lambda device: 77)
        assert both() == (4, 6)
        print("DONE")
    """)


@pytest.mark.parametrize("bad", [
    "({}, device, stream)", "(without_last, device, stream)", "(dict(new, dg_grad_norm=0), device, stream)",
    "(dict(new, dg_grad_norm='here'), device, stream)", "(dict(new, dg_grad_norm=-1), device, stream)",
    "(dict(new, dg_grad_norm=1 << 70), device, stream)", "(new, None, stream)", "(new, device, 7)", "(new,)",
    "(list(new), device, stream)"])
def test_a_failed_init_leaves_the_calls_as_they_were(bad):
    run(f"""
        native.init(table(3, 5), lambda: 0, lambda device: 77)
        new, device, stream = table(8, 9), lambda: 1, lambda device: 99
        without_last = {{n: a for n, a in new.items() if n != "dg_grad_clip"}}
        try:
            native.init(*{bad})
        except (TypeError, ValueError, OverflowError):
            pass
        else:
            raise AssertionError("init took it")
        assert both() == (3, 5)
        print("DONE")
    """)


def test_without_init_no_call_is_made():
    run("""
        assert both() == (None, None)
        print("DONE")
    """)
