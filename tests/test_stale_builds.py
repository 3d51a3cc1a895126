"""Libraries that do not belong to the sources beside them are refused with a
message that says what to do."""
import shutil
import subprocess

import pytest

from query_aware_sparse_tb_b200 import _lib


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
