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


def calls():
    """Every call of the native binding with arguments whose types and shapes are in order."""
    f32, bf, i32 = torch.float32, torch.bfloat16, torch.int32
    z = lambda *s, t=f32: torch.zeros(*s, dtype=t)  # noqa: E731
    q, k, c, mask, b, one = z(2, 4, 64), z(2, 2, 64), z(2, 16, 64, t=bf), z(2, 1, t=i32), z(2, t=i32), z(1, t=i32)
    ws = z(4096, t=torch.uint8)
    caches = nt.pointer_array([c, c])
    return {
        "nt_rope_frequencies": (lambda: nt.nt_rope_frequencies(64, 1e4, z(32, t=torch.float64), stream=0)),
        "nt_qk_norm_rope_append": lambda **x: nt.nt_qk_norm_rope_append(q, k, k, None, None, 1e-6, z(32, t=torch.float64), 0, 1.0, q, c, c,
                                                                        **{"n_bad": one, "stream": 0, **x}),
        "nt_tree_layout": lambda **x: nt.nt_tree_layout(b, mask, b, **{"n_bad": one, "stream": 0, **x}),
        "nt_tree_attention": lambda **x: nt.nt_tree_attention(q, c, c, 4, 4, mask, q, ws, **{"stream": 0, **x}),
        "nt_token_counts": lambda **x: nt.nt_token_counts(b, z(9, t=i32), **{"n": one, "n_bad": one, "stream": 0, **x}),
        "nt_logits_adjust": lambda **x: nt.nt_logits_adjust(z(2, 9), argmax=b, ws=ws, **{"stream": 0, **x}),
        "nt_tree_accept": lambda **x: nt.nt_tree_accept(b, b, b, b, b, x.pop("n_emit", one), **{"stream": 0, **x}),
        "nt_tree_commit": lambda **x: nt.nt_tree_commit(caches, caches, 2, 64, 16, b, x.pop("n_emit", one), 4, 4, **{"stream": 0, **x}),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_tensors_of_the_host_are_refused(name):
    with pytest.raises(nt.NtError, match="must be a CUDA tensor") as e:
        calls()[name]()
    assert e.value.status == nt.NT_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["nt_tree_attention", "nt_logits_adjust", "nt_tree_accept"])
def test_tensors_of_the_host_are_refused_on_the_current_stream_too(name):
    with pytest.raises(nt.NtError, match="must be a CUDA tensor"):
        calls()[name](stream=None)


@pytest.mark.parametrize("name,which", [("nt_qk_norm_rope_append", "n_bad"), ("nt_tree_layout", "n_bad"), ("nt_token_counts", "n"),
                                        ("nt_token_counts", "n_bad"), ("nt_tree_accept", "n_emit"), ("nt_tree_commit", "n_emit")])
def test_a_number_needs_an_element(name, which):
    """An empty tensor has no address and passed for one that was left out: nt_token_counts then had no bound."""
    with pytest.raises(nt.NtError, match=f"{which} must have an element") as e:
        calls()[name](**{which: torch.zeros(0, dtype=torch.int32)})
    assert e.value.status == nt.NT_ERR_INVALID_ARG


def test_a_stream_that_is_no_address_is_a_python_error():
    # (reached behind the check of the tensors on a machine with a GPU)
    with pytest.raises((OverflowError, nt.NtError)):
        calls()["nt_tree_accept"](stream=1 << 80)
