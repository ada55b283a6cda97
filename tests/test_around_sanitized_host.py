"""The host side of the operators around the products (argument checks, sizes,
error messages) under AddressSanitizer and UndefinedBehaviorSanitizer on the host
code only, in a subprocess that preloads the ASan runtime.  No GPU: every call
returns before any HIP call."""
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "moe_grouped_gemm_nt_amd")
SOURCES = ["dg_api", "route", "expert_rows", "lora"]

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
    each("dg_route_topk", [P, 0, P, P, P, 4, 64, 8, 0, 8, 4, 2, 1, f, None],
         {0: [None, B], 1: [-1, 2, big], 2: [B], 3: [None, B], 4: [None, B], 5: [-1, low], 6: [0, low, big], 7: [0, big],
          8: [2, -1], 9: [0, 7, big, low], 10: [0, 9, low], 11: [0, 3]})
    each("dg_route_topk_backward", [P, 0, P, P, P, 4, 64, 8, 0, 1, f, None],
         {0: [None, B], 1: [2], 2: [None, B], 3: [None, B], 4: [None, B], 5: [-1, low], 6: [0, big], 7: [0, 65], 8: [2]})
    each("dg_m_grouped_layout_contiguous", [P, 4, 2, 0, 8, 128, P, P, P, P, None],
         {0: [None, B], 1: [-1, low, big], 2: [0, big, low], 4: [0, low, big], 5: [100, low, -128], 6: [None, B],
          7: [None, B], 8: [None, B], 9: [B]})
    each("dg_m_grouped_layout_masked", [P, 4, 2, 0, 8, 16, P, P, P, None],
         {0: [None, B], 1: [-1, low, big], 2: [0, big, low], 4: [0, low, big], 5: [-1, low, big], 6: [None, B],
          7: [None, B], 8: [None, B]})
    each("dg_m_grouped_scatter_fp8_contiguous", [P, P, P, P, P, P, 4, 2, 128, 256, 0, None],
         {0: [None, B], 1: [B], 2: [None, B], 3: [None, B], 4: [None, B], 5: [None, B], 6: [-1, low, big],
          7: [0, low, big], 8: [-1, low], 9: [-128, 100, low, big]})
    each("dg_m_grouped_scatter_fp8_masked", [P, P, P, P, P, P, 4, 2, 4, 16, 256, 0, None],
         {0: [None, B], 1: [B], 2: [None, B], 3: [None, B], 4: [None, B], 5: [None, B], 6: [-1, low, big],
          7: [0, low, big], 8: [0, low, big], 9: [-1, low, big], 10: [-128, 100, low, big]})
    each("dg_k_grouped_scatter_fp8", [P, P, P, P, P, 4, 2, 256, 64, 0, None],
         {0: [None, B], 1: [B], 2: [None, B], 3: [None, B], 4: [None, B], 5: [-1, low, big], 6: [0, low, big],
          7: [-128, 100, low, big], 8: [-16, 72, low, big]})
    each("dg_m_grouped_gather", [P, P, P, P, P, 4, 2, 128, 65, None],
         {0: [None, ctypes.c_void_p(1)], 1: [None, B], 2: [B], 3: [ctypes.c_void_p(1)], 4: [None, ctypes.c_void_p(1)],
          5: [-1, low, big], 6: [0, 65, low, big], 7: [-1, low], 8: [-1, low]})
    each("dg_m_grouped_gather_weight_grad", [P, P, P, P, 4, 2, 128, 65, None],
         {0: [None, ctypes.c_void_p(1)], 1: [None, B], 2: [None, ctypes.c_void_p(1)], 3: [None, B], 4: [-1, low, big],
          5: [0, 65, low, big], 6: [-1, low], 7: [-1, low]})
    each("dg_lora_bf16_nt", [P, 256, P, P, P, P, P, 65, P, 65, 4, 65, 256, 16, 3, None],
         {0: [None, B], 1: [255, 260, low], 2: [None, B], 3: [None, B], 4: [B], 5: [None, B], 6: [ctypes.c_void_p(1)],
          7: [64, 66, low], 8: [None, ctypes.c_void_p(1)], 9: [64, 66, low], 10: [-1, low], 11: [-1, low, big],
          12: [-128, 100, low, big], 13: [-8, 12, 264, low], 14: [-1, 1025, low, big]})
    bound = lib.dg_m_grouped_rows_bound
    bound.argtypes = [ctypes.c_longlong, ctypes.c_int]
    for n, g in itertools.product([-1, 0, 1, 127, 128, 10**6, 2**30, 2**31 - 1, 2**31, 2**62, -2**62], [-1, 0, 1, 7, 1024, big]):
        r = bound(n, g)
        calls += 1
        assert r == -1 or (r >= 0 and r % 128 == 0 and (g == 0 or r >= n)), (n, g, r)
    print(f"SANITIZED_OK {calls}")
""")


@pytest.fixture(scope="module")
def sanitized_lib(tmp_path_factory):
    from moe_grouped_gemm_nt_amd import build
    kernels = [os.path.join(PKG, "_build", f) for f in ("fp8_gemm.o", "fp8_gemm_e8m0.o")]
    if not all(os.path.exists(k) for k in kernels):
        build.build()
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    out = tmp_path_factory.mktemp("asan_around")
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
