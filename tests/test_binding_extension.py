"""The binding's extension is built for one torch and Python, and nothing but
the host time of a call depends on it."""
import os
import subprocess
import sys

import torch

from mx_microscaling_mixed_b200 import build


def test_it_is_built_and_loaded_here():
    build.build()
    from mx_microscaling_mixed_b200 import capi
    assert capi._binding is not None and capi._binding.__file__ == build.binding_path()


def test_another_torch_takes_another_file(monkeypatch):
    build.build()
    here = build.binding_path()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    other = build.binding_path()
    assert other != here and not os.path.exists(other) and build._stale(other, [])
    monkeypatch.undo()
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert build.binding_path() != here


def test_every_entry_point_is_there_without_it():
    code = """
from mx_microscaling_mixed_b200 import build
build.binding_path = lambda: "/nonexistent/extension.so"
from mx_microscaling_mixed_b200 import capi as c
assert c._binding is None
assert all(hasattr(c._lib, n) for n in c.EXPORTS)
c.mxs_rope_plan(64)
lay = c.mxs_layout_make(128, (0, 0, 128))
cache = c.kv_cache_empty(4, 2, 64, device="cpu")
import torch
x = torch.zeros(4, 2, 64)
for call in (lambda: c.mxs_rope(x, torch.arange(4), c.mxs_rope_plan(64)), lambda: c.mxs_kv_write(x, x, cache, torch.arange(4)),
             lambda: c.mxs_kv_read(cache, torch.arange(4))):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)


def test_the_library_is_built_where_it_cannot_be(monkeypatch, tmp_path, capfd):
    build.build()
    path = tmp_path / "_binding-of-a-torch-without-headers.so"
    monkeypatch.setattr(build, "binding_path", lambda: str(path))
    monkeypatch.setattr(build, "OBJ", str(tmp_path))
    monkeypatch.setenv("CXX", "false")
    assert build.build() == build.LIB and not path.exists()
    assert "not built" in capfd.readouterr().err
