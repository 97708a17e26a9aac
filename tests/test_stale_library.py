"""A library built before the binding is refused in words, whichever of its functions are missing."""
import shutil
import subprocess

import pytest

import reduction_codec_amd as rca

OLDER = """
#include <stddef.h>
int rc_abi_version(void) { return VERSION; }
size_t rc_tile_bytes(int a, int b, int c) { return 0; }
"""


@pytest.fixture
def library(tmp_path, monkeypatch):
    def build(source, **defines):
        src, lib = tmp_path / "older.c", tmp_path / "older.so"
        src.write_text(source)
        subprocess.run(["gcc", "-shared", "-fPIC", *[f"-D{k}={v}" for k, v in defines.items()], str(src), "-o", str(lib)],
                       check=True)
        monkeypatch.setattr(rca, "LIB_PATH", str(lib))
        monkeypatch.setattr(rca, "_lib", None)
    return build


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("source,version,says", [
    (OLDER, rca.ABI_VERSION, "older than this binding.*rebuild"), (OLDER, rca.ABI_VERSION - 1, "ABI version 2.*rebuild"),
    ("int nothing;", 0, "older than this binding.*rebuild")])
def test_older_library(library, source, version, says):
    library(source, VERSION=version)
    with pytest.raises(RuntimeError, match=says):
        rca.lib()
    assert rca._lib is None
