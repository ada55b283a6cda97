"""The library without the native side of its Python binding: libdg.so is built where torch, its headers, Python's or
g++ are missing, and the calls then go through ctypes, with the same checks."""
import os
import shutil
import sys

import pytest
import torch

import moe_grouped_gemm_nt_amd as dg
import moe_grouped_gemm_nt_amd._lib as lib
from moe_grouped_gemm_nt_amd import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Everything is built in a folder of its own, by a compiler that only writes its output's name into it; a
    _binding.so of an earlier build lies there.  (the folder, the commands)"""
    commands = []

    def compiler(cmd, verbose):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")

    monkeypatch.setattr(build, "_run", compiler)
    monkeypatch.setattr(build, "PKG_DIR", str(tmp_path))
    for name, file in (("LIB_PATH", "libdg.so"), ("BINDING_PATH", "_binding.so"), ("CEILINGS_PATH", "libdg_ceilings.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    (tmp_path / "_binding.so").write_text("earlier")
    return tmp_path, commands


def without_compiler(monkeypatch):
    which = shutil.which
    monkeypatch.setattr(shutil, "which", lambda c: None if c in ("g++", "c++") else which(c))


def without_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)


def without_headers(monkeypatch):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nowhere"})


@pytest.mark.skipif(build.binding_lacks() is not None, reason="the native side cannot be built here")
def test_all_there(tree):
    folder, commands = tree
    assert build.build() == str(folder / "libdg.so")
    assert (folder / "libdg.so").read_text() == (folder / "_binding.so").read_text() == "built"
    assert sum("binding.cpp" in " ".join(c) for c in commands) == 1


@pytest.mark.parametrize("missing", [without_compiler, without_torch, without_headers], ids=lambda f: f.__name__)
def test_the_library_is_built_without(tree, monkeypatch, capsys, missing):
    folder, commands = tree
    missing(monkeypatch)
    build.build()
    assert (folder / "libdg.so").read_text() == (folder / "libdg_ceilings.so").read_text() == "built"
    assert not any("binding.cpp" in " ".join(c) for c in commands)
    assert not (folder / "_binding.so").exists()               # one of other sources must not stay
    assert "_binding.so" in capsys.readouterr().err


@pytest.mark.skipif(build.binding_lacks() is not None, reason="the native side cannot be built here")
def test_an_error_in_the_binding_is_raised_after_the_library(tree, monkeypatch):
    folder, _ = tree
    compiler = build._run

    def failing(cmd, verbose):
        if "binding.cpp" in " ".join(cmd):
            raise RuntimeError("g++ failed")
        compiler(cmd, verbose)

    monkeypatch.setattr(build, "_run", failing)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert (folder / "libdg.so").read_text() == "built" and not (folder / "_binding.so").exists()


@pytest.fixture
def no_native(monkeypatch):
    monkeypatch.setattr(lib, "_native", None)
    monkeypatch.delattr(dg, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, dg.__name__ + "._binding", None)


BF = torch.bfloat16
CALLS = [
    (lambda: dg.dg_route_balance(torch.zeros(2, 4), torch.zeros(2, 1), None, torch.zeros(1), torch.zeros(1, 4)), "topk_ids"),
    (lambda: dg.dg_route_balance_backward(torch.zeros(2, 4), torch.zeros(1, 4), None, None, None, torch.zeros(2, 4), 1),
     "counts"),
    (lambda: dg.dg_bf16_fp4_gemv_nt(torch.zeros(2, 128, dtype=BF), torch.zeros(4, 64), None, None, None), "d must be"),
    (lambda: dg.dg_grad_norm([torch.zeros(3)], torch.zeros(2)), "norm"),
    (lambda: dg.dg_grad_clip([torch.zeros(3)], [torch.zeros(4)], torch.zeros(1), 1.0), "types and sizes"),
]


@pytest.mark.parametrize("call,named", CALLS, ids=[c[1] for c in CALLS])
def test_the_calls_check_their_arguments_without_it(no_native, call, named):
    with pytest.raises((ValueError, TypeError), match=named):
        call()
    assert lib._load_native() is False


def test_a_binding_that_cannot_be_loaded_is_named(no_native, monkeypatch, tmp_path):
    file = tmp_path / "_binding.so"
    file.write_text("of another torch")
    monkeypatch.setattr(lib, "BINDING_PATH", str(file))
    with pytest.warns(RuntimeWarning, match="_binding.so"):
        assert lib._load_native() is False


def test_a_missing_one_is_no_warning(no_native, monkeypatch, tmp_path, recwarn):
    monkeypatch.setattr(lib, "BINDING_PATH", str(tmp_path / "_binding.so"))
    assert lib._load_native() is False and not recwarn.list
