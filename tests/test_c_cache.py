"""The paged cache's C ABI from a strict C99 program, tests/abi_cache.c: the struct's layout, and that the binding
fills it in word by word as C lays it out."""
import os
import shutil
import subprocess

import pytest
import torch

import reduction_codec_amd as rca
from tests.test_c_consumer import LIB, LIBDIR, ROOT


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_c_program_uses_the_cache(tmp_path):
    assert os.path.exists(LIB), "build the library first (__graft_entry__.build())"
    exe = tmp_path / "abi_cache"
    cmd = ["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
           os.path.join(ROOT, "tests", "abi_cache.c"), "-o", str(exe), LIB, f"-Wl,-rpath,{LIBDIR}",
           "-Wl,-rpath-link,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all checks held" in r.stdout


def test_the_bindings_words(monkeypatch):
    monkeypatch.setattr(rca, "_check_dev", lambda *a: None)
    monkeypatch.setattr(rca, "_check_on", lambda *a: None)
    k, v = rca.mxfp4_cache_new(5, 3, 32, 128, "cpu")
    table, lengths, offsets = (torch.zeros(n, dtype=torch.int32) for n in ((2, 7), (2,), (3,)))
    words = rca._cache(k, v, table, lengths, offsets, 128, None)
    assert words.itemsize * len(words) == 88
    assert words.tolist() == [k.data_ptr(), v.data_ptr(), 5, 32, 3, 128, table.data_ptr(), 2, 7, lengths.data_ptr(),
                              offsets.data_ptr()]
