"""The library and the native part of its Python binding: who needs which, and what the binding refuses (no GPU needed)."""
import os
import subprocess
import sys

import pytest
import torch

from packed_weight_gemv_gb300 import build as nt_build
from packed_weight_gemv_gb300 import nt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    nt_build.build()


@pytest.mark.parametrize("binding", ["missing", "stale"])
def test_calls_of_the_library_alone_need_no_native_binding(binding, tmp_path):
    path = tmp_path / "_ntbind.so"
    if binding == "stale":  # what cannot be imported, as after a change of torch or Python
        path.write_bytes(b"not a module of this Python")
    prog = f"""
from packed_weight_gemv_gb300 import nt
nt.BIND_PATH = {str(path)!r}
assert nt.nt_repack_size(128, 512) > 0 and nt.load_library().nt_abi_version() == 1
import torch
i = torch.zeros(1, dtype=torch.int32)
try:
    nt.nt_tree_layout(i, i.view(1, 1), stream=0)
except RuntimeError as e:
    print("refused:", e)
"""
    r = subprocess.run([sys.executable, "-c", prog], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.startswith("refused:") and str(path) in r.stdout and "build" in r.stdout


def test_the_binding_is_built_again_for_another_torch_or_python(monkeypatch, tmp_path):
    assert nt_build.binding_is_current()
    monkeypatch.setattr(nt_build.sys, "version", "3.99.0")
    assert not nt_build.binding_is_current()
    monkeypatch.undo()
    assert nt_build.binding_is_current()
    monkeypatch.setattr(nt_build.importlib.metadata, "version", lambda name: "0.0")
    assert not nt_build.binding_is_current()
    monkeypatch.undo()
    monkeypatch.setattr(nt_build, "BIND_STAMP", str(tmp_path / "none"))
    assert not nt_build.binding_is_current()
