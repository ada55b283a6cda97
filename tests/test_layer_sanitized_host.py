"""The host side of the balance loss, the 4-bit products and the gradients' calls
(argument checks, sizes, lists of tensors, error messages) under AddressSanitizer
and UndefinedBehaviorSanitizer on the host code only, in a subprocess that preloads the ASan runtime.  No GPU: every call
returns before any HIP call."""
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "moe_grouped_gemm_nt_amd")
SOURCES = ["dg_api", "expert_rows", "balance", "gemv4", "grads"]

DRIVER = textwrap.dedent(r"""
    import ctypes, itertools, sys
    lib = ctypes.CDLL(sys.argv[1])
    lib.dg_last_error.restype = ctypes.c_char_p
    P = ctypes.c_void_p(0x100000)             # aligned, never read
    B = ctypes.c_void_p(0x100002)             # aligned to 2
    f = ctypes.c_float(1.0)
    calls = 0

    def each(name, good, bad):
        # every argument replaced in turn by each of its bad values
        global calls
        fn = getattr(lib, name)
        for at, values in bad.items():
            for v in values:
                args = list(good)
                args[at] = v
                rc = fn(*args)
                calls += 1
                assert rc in (-1, -2), (name, at, v, rc)
                assert lib.dg_last_error(), (name, at, v)

    big, low = 2**31 - 1, -2**31
    Q = ctypes.c_void_p(0x900000)
    O = ctypes.c_void_p(1)
    each("dg_route_balance", [P, 0, P, P, P, P, 4, 64, 8, 3, 1, f, None],
         {0: [None, B], 1: [-1, 2, big], 2: [None, B], 3: [None, B], 4: [None, B], 5: [None, B], 6: [-1, low, big],
          7: [0, low, big], 8: [0, 65, big], 9: [-1, low], 10: [2, -1]})
    each("dg_route_balance_backward", [P, 0, P, P, P, P, P, 4, 64, 8, 3, 1, f, None],
         {0: [None, B], 1: [2], 2: [None, B], 3: [None, B], 4: [B], 5: [B], 6: [None, B], 7: [-1, low, big],
          8: [0, low, big], 9: [0, 65, big], 10: [-1, low], 11: [2, -1]})
    each("dg_bf16_fp4_gemv_nt", [P, 256, P, P, P, 65, Q, 65, 4, 65, 256, None],
         {0: [None, B], 1: [255, 260, low], 2: [None, B], 3: [None, B], 4: [O], 5: [64, low], 6: [None, O], 7: [64, low],
          8: [-1, low], 9: [-1, low, big], 10: [-128, 100, low, big]})
    each("dg_bf16_int4_gemv_nt", [P, 256, P, P, 0, P, 64, P, 65, Q, 65, 4, 65, 256, None],
         {0: [None, B], 1: [255, 260, low], 2: [None, B], 3: [None, B], 4: [2, -1], 6: [0, 16, 256, low], 7: [O],
          8: [64, low], 9: [None, O], 10: [64, low], 11: [-1, low], 12: [-1, low, big], 13: [-128, 100, low, big]})
    each("dg_m_grouped_bf16_fp4_gemv_nt_topk", [P, 256, 4, P, P, P, P, 65, Q, 65, 4, 2, 0, 3, 65, 256, None],
         {0: [None, B], 1: [255, 260, low], 2: [5, low, big], 3: [None, B], 4: [None, B], 5: [None, B], 6: [O],
          7: [64, low], 8: [None, O], 9: [64, low], 10: [-1, low, big], 11: [0, low, big], 12: [-1, low],
          13: [-1, 1025, low, big], 14: [-1, low, big], 15: [-128, 100, low, big]})
    each("dg_m_grouped_bf16_int4_gemv_nt_topk", [P, 256, 8, P, P, P, 1, None, 32, P, 65, Q, 65, 4, 2, 0, 3, 65, 256, None],
         {0: [None, B], 1: [255, 260, low], 2: [5, low, big], 3: [None, B], 4: [None, B], 5: [None, O], 6: [2, -1],
          8: [0, 96, low], 9: [O], 10: [64, low], 11: [None, O], 12: [64, low], 13: [-1, low, big], 14: [0, low, big],
          15: [-1, low], 16: [-1, 1025, low, big], 17: [-1, low, big], 18: [-128, 100, low, big]})

    def lists(pointers, types, sizes):
        n = len(pointers)
        return (ctypes.c_void_p * n)(*pointers), (ctypes.c_int * n)(*types), (ctypes.c_longlong * n)(*sizes)

    p, t, s = lists([0x100000, 0x200000, 0x300000], [0, 1, 0], [100, 0, 7])
    o = lists([0x500000, 0x600000, 0x700000], [0, 1, 0], [100, 0, 7])[0]
    bad_p = [None, lists([0, 1, 2], t, s)[0], lists([0x100002, 0, 0x300000], t, s)[0]]
    bad_t = [None] + [lists(p, v, s)[1] for v in ([2, 1, 0], [0, 1, -1], [0, big, 0])]
    bad_s = [None] + [lists(p, t, v)[2] for v in ([-1, 0, 0], [0, -2**63, 0], [0, 0, 2**43 + 1], [0, 2**63 - 1, 0])]
    each("dg_grad_norm", [p, t, s, 3, P, None], {0: bad_p, 1: bad_t, 2: bad_s, 3: [-1, low, big], 4: [None, B]})
    same = lists([0x500000, 0x500000, 0x500004], t, s)[0]
    part = lists([0x100004, 0x600000, 0x700000], t, s)[0]
    most = ctypes.c_float(1.0)
    each("dg_grad_clip", [p, o, t, s, 3, Q, most, None],
         {0: bad_p, 1: bad_p + [same, part], 2: bad_t, 3: bad_s, 4: [-1, low, big], 5: [None, B, ctypes.c_void_p(0x500018)],
          6: [ctypes.c_float(-1.0), ctypes.c_float(float("nan")), ctypes.c_float(float("-inf"))]})
    # many tensors, none of them apart: sorted on the host
    n = 1 << 15
    many = lists([0x100000 + 4 * (i * 7919 % n) for i in range(n)], [0] * n, [2] * n)
    assert lib.dg_grad_clip(many[0], many[0], many[1], many[2], n, Q, most, None) == -1
    print(f"SANITIZED_OK {calls}")
""")


@pytest.fixture(scope="module")
def sanitized_lib(tmp_path_factory):
    from moe_grouped_gemm_nt_amd import build
    kernels = [os.path.join(PKG, "_build", f) for f in ("fp8_gemm.o", "fp8_gemm_e8m0.o")]
    if not all(os.path.exists(k) for k in kernels):
        build.build()
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    out = tmp_path_factory.mktemp("asan_layer")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = [f for f in build.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"]
    procs = []
    for s in SOURCES:
        procs.append((str(out / f"{s}.o"), subprocess.Popen(
            [hipcc] + flags + san + ["-I", os.path.join(ROOT, "include"), "-c", os.path.join(PKG, "csrc", s + ".hip"),
                                     "-o", str(out / f"{s}.o")], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
            text=True)))
    for _, p in procs:
        text, _ = p.communicate()
        assert p.returncode == 0, text[-3000:]
    lib = str(out / "libdg_san.so")
    r = subprocess.run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC"] + san + [o for o, _ in procs] + kernels +
                       ["-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    rt = subprocess.run([hipcc, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True,
                        text=True).stdout.strip()
    assert os.path.exists(rt), rt
    return lib, rt


def test_argument_checks_under_address_and_undefined_behaviour_sanitizers(sanitized_lib, tmp_path):
    lib, rt = sanitized_lib
    script = tmp_path / "drive.py"
    script.write_text(DRIVER)
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, str(script), lib], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "SANITIZED_OK" in r.stdout, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
