"""Libraries that do not belong to the sources beside them are refused with a
message that says what to do."""
import os
import shutil
import subprocess
import types

import pytest

import query_aware_sparse_tb_b200 as package
from query_aware_sparse_tb_b200 import _lib, build


def c_library(tmp_path, source):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, lib = tmp_path / "old.c", tmp_path / "libtb.so"
    src.write_text(source)
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True, capture_output=True, text=True)
    return str(lib)


@pytest.mark.parametrize("source,message", [
    (f"int tb_abi_version(void) {{ return {_lib.TB_ABI_VERSION}; }}", "lacks .*tb_tree_accept.*rebuild"),
    (f"int tb_abi_version(void) {{ return {_lib.TB_ABI_VERSION - 1}; }}",
     f"ABI version {_lib.TB_ABI_VERSION - 1}, .*rebuild"),
    ("int other(void) { return 0; }", "tb_abi_version.*rebuild"),
])
def test_a_library_of_older_sources_is_refused_with_a_message(tmp_path, source, message):
    with pytest.raises(_lib.TbError, match=message):
        _lib.load(c_library(tmp_path, source))


# ------------------------------------------------------------------ the call module

@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """build_call() with a compiler that only notes that it was called, into a
    folder of its own."""
    runs, script = tmp_path / "runs", tmp_path / "cxx"
    script.write_text(f'#!/bin/sh\necho "$@" >> {runs}\nwhile [ "$1" != "-o" ]; do shift; done\ntouch "$2"\n')
    script.chmod(0o755)
    monkeypatch.setattr(build, "CXX", str(script))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "_tbcall.so"))
    return lambda: len(runs.read_text().splitlines()) if runs.exists() else 0


def test_the_call_module_is_built_again_for_another_torch(compiler, monkeypatch):
    build.build_call()
    build.build_call()
    assert compiler() == 1                        # nothing changed
    monkeypatch.setattr(build, "call_tag", lambda: "torch 1.0, cpython-39")
    build.build_call()
    build.build_call()
    assert compiler() == 2
    os.utime(build.CALL, (0, 0))                  # older than its sources
    build.build_call()
    assert compiler() == 3


def test_the_library_is_built_without_a_cpp_compiler(compiler, monkeypatch):
    build.build_call()
    monkeypatch.setattr(build, "CXX", "/no/such/compiler")
    monkeypatch.setattr(build, "call_tag", lambda: "torch 1.0, cpython-39")
    with pytest.raises(OSError):
        build.build_call()
    assert not os.path.exists(build.CALL)         # the stale one is gone
    monkeypatch.setattr(build, "SOURCES", [])     # (nothing to compile)
    monkeypatch.setattr(build, "LIB", os.path.join(build.BUILD, "libtb.so"))
    open(build.LIB, "w").close()
    with pytest.warns(UserWarning, match="libtb.so is built, _tbcall.so is not"):
        assert build.build() == build.LIB


def test_a_call_module_of_another_torch_is_refused(monkeypatch):
    build.build()
    monkeypatch.setattr(_lib, "_call", None)
    for fake in (types.SimpleNamespace(built_for="torch 1.0, cpython-39"), types.SimpleNamespace()):
        monkeypatch.setattr(package, "_tbcall", fake, raising=False)
        with pytest.raises(_lib.TbError, match="built for .*rebuild"):
            _lib._tbcall()
        assert _lib._call is None


def test_the_call_module_shares_the_cpp_runtime_of_torch(monkeypatch):
    """With a C++ runtime of its own (as a compiler that links it statically
    gives) the module's error messages crashed the process."""
    if shutil.which("readelf") is None:
        pytest.skip("readelf not available")
    monkeypatch.setenv("CXX", "/no/such/compiler")  # not the environment's choice
    build.build_call(force=True)
    needed = subprocess.run(["readelf", "-d", build.CALL], check=True, capture_output=True, text=True).stdout
    assert "libstdc++.so.6" in needed
