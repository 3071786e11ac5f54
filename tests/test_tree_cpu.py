"""Refusals of the tree-verify calls: every malformed argument is answered on the host before any
launch (no GPU needed), with the status the header states; well-formed ones get as far as the
device check."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import build as nt_build
from packed_weight_gemv_gb300 import nt
from tests import _tree

INV, ALIGN, UNSUP, WS = nt.NT_ERR_INVALID_ARG, nt.NT_ERR_ALIGNMENT, nt.NT_ERR_UNSUPPORTED, nt.NT_ERR_WORKSPACE
P = [0x100000 * (i + 1) for i in range(12)]  # addresses that are never read


@pytest.fixture(scope="module")
def lib():
    nt_build.build()
    return nt.load_library()


def call(fn, good, **bad):
    return fn(*[bad.get(k, v) for k, v in good.items()])


def reaches_device(status):
    """Past every argument check: the device check answers (there is no GPU here)."""
    return status in (nt.NT_OK, nt.NT_ERR_UNSUPPORTED, nt.NT_ERR_CUDA)


APPEND = dict(q=P[0], k=P[1], v=P[2], dtype=0, qs=512, ks=256, vs=256, qg=P[3], kg=P[4], eps=1e-6, B=3, Hq=4, Hkv=2,
              D=128, f=P[5], rd=64, layout=0, amp=1.0, pos=None, pos0=7, rows=None, row0=5, q_out=P[6], kc=P[7], vc=P[8],
              ts=64, n_bad=None, stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(q_out=None), INV), (dict(kc=None), INV),
    (dict(vc=None), INV), (dict(f=None), INV), (dict(dtype=2), INV), (dict(dtype=-1), INV), (dict(layout=2), INV),
    (dict(D=124), UNSUP), (dict(D=264), UNSUP), (dict(D=0), UNSUP), (dict(rd=4), INV), (dict(rd=136), INV), (dict(rd=-8), INV),
    (dict(B=0), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(Hq=65536), INV), (dict(ts=0), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(pos0=2 ** 31 - 2), INV), (dict(row0=-1), INV), (dict(row0=62), INV),
    (dict(row0=2 ** 31 - 1), INV), (dict(qs=510), ALIGN), (dict(ks=258), ALIGN), (dict(vs=1), ALIGN), (dict(qs=508), INV),
    (dict(ks=252), INV), (dict(vs=-256), INV), (dict(q=P[0] + 8), ALIGN), (dict(q=P[0] + 4, dtype=1), ALIGN),
    (dict(q_out=P[6] + 8), ALIGN), (dict(kc=P[7] + 2), ALIGN), (dict(qg=P[3] + 4), ALIGN), (dict(f=P[5] + 4), ALIGN),
    (dict(pos=P[9] + 2), ALIGN), (dict(rows=P[9] + 1), ALIGN), (dict(n_bad=P[9] + 1), ALIGN)])
def test_append_refusals(lib, bad, status):
    assert call(lib.nt_qk_norm_rope_append, APPEND, **bad) == status


def test_well_formed_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real: only where there is no device")
    for ok in (dict(), dict(q=P[0] + 8, dtype=1), dict(pos=P[9], pos0=2 ** 31 - 1), dict(rows=P[9], row0=-5),
               dict(rd=0, f=None), dict(qg=None, kg=None), dict(B=1, qs=0)):
        assert reaches_device(call(lib.nt_qk_norm_rope_append, APPEND, **ok)), ok
    for fn, good in ((lib.nt_tree_attention, ATTEND), (lib.nt_logits_adjust, ADJUST), (lib.nt_tree_layout, LAYOUT),
                     (lib.nt_tree_accept, ACCEPT), (lib.nt_tree_commit, commit_args()), (lib.nt_token_counts, COUNTS)):
        assert reaches_device(call(fn, good))


FREQ = dict(rd=64, base=1e4, scaling=2, factor=4.0, trained=4096, slow=1.0, fast=32.0, out=P[0], stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(out=None), INV), (dict(rd=0), INV), (dict(rd=12), INV), (dict(rd=264), INV), (dict(base=1.0), INV),
    (dict(base=float("nan")), INV), (dict(base=float("inf")), INV), (dict(scaling=3), INV), (dict(factor=0.0), INV),
    (dict(scaling=1, factor=-1.0), INV), (dict(trained=0), INV), (dict(slow=-1.0), INV), (dict(slow=32.0), INV),
    (dict(fast=float("nan")), INV), (dict(out=P[0] + 4), ALIGN)])
def test_frequency_refusals(lib, bad, status):
    assert call(lib.nt_rope_frequencies, FREQ, **bad) == status


ATTEND = dict(q=P[0], dtype=0, kc=P[1], vc=P[2], B=5, Hq=8, Hkv=2, D=128, prefix=100, row0=100, ts=128, mask=P[3], words=1,
              out=P[4], ws=P[5], ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INV), (dict(kc=None), INV), (dict(vc=None), INV), (dict(mask=None), INV), (dict(out=None), INV),
    (dict(dtype=2), INV), (dict(D=96), UNSUP), (dict(D=256), UNSUP), (dict(B=0), INV), (dict(B=257, words=9, ts=512), INV),
    (dict(Hkv=0), INV), (dict(Hq=1), INV), (dict(Hq=9), INV), (dict(words=0), INV), (dict(B=33, ts=512), INV),
    (dict(prefix=-1), INV), (dict(row0=99), INV), (dict(row0=124), INV), (dict(row0=2 ** 31 - 1), INV),
    (dict(Hq=2 ** 20), INV), (dict(q=P[0] + 8), ALIGN), (dict(kc=P[1] + 8), ALIGN), (dict(vc=P[2] + 2), ALIGN),
    (dict(out=P[4] + 4), ALIGN), (dict(mask=P[3] + 2), ALIGN), (dict(ws=None), WS), (dict(ws=P[5] + 8), WS),
    (dict(ws_bytes=0), WS)])
def test_attention_refusals(lib, bad, status):
    assert call(lib.nt_tree_attention, ATTEND, **bad) == status


def test_attention_workspace_does_not_depend_on_the_prefix(lib):
    for shape in ((1, 32, 8, 128), (40, 160, 160, 64), (255, 32, 4, 64), (256, 64, 64, 128)):
        assert len({nt.nt_tree_attention_workspace_size(*shape, p) for p in (0, 1, 64, 1000, 2000, 30000, 1 << 20)}) == 1


def test_attention_workspace_is_what_the_call_wants(lib):
    for B, Hq, Hkv, D, prefix in ((5, 8, 2, 128, 100), (1, 32, 8, 128, 30000), (256, 32, 4, 64, 16000), (1, 1, 1, 64, 0)):
        n = nt.nt_tree_attention_workspace_size(B, Hq, Hkv, D, prefix)
        a = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, prefix=prefix, row0=prefix, ts=prefix + B, words=(B + 31) // 32)
        assert n >= 16 and call(lib.nt_tree_attention, ATTEND, **a, ws_bytes=n - 1) == WS
    for bad in ((0, 8, 2, 128, 1), (257, 8, 2, 128, 1), (1, 9, 2, 128, 1), (1, 8, 0, 128, 1), (1, 8, 2, 128, -1), (1, 8, 2, 32, 1)):
        with pytest.raises(nt.NtError):
            nt.nt_tree_attention_workspace_size(*bad)


ADJUST = dict(x=P[0], B=2, V=100, counts=P[1], cs=0, tm=P[2], words=1, tok=P[3], rep=1.1, freq=0.1, pres=0.1, bias=P[4],
              bs=100, al=P[5], als=4, out=P[6], am=P[7], ws=P[8], ws_bytes=4096, stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), INV), (dict(out=None, am=None), INV), (dict(B=0), INV), (dict(B=65536), INV), (dict(V=0), INV),
    (dict(V=2 ** 31 - 1), INV), (dict(tok=None), INV), (dict(tm=None), INV), (dict(words=0), INV), (dict(B=257, words=9), INV),
    (dict(rep=0.0), INV), (dict(rep=-1.0), INV), (dict(rep=float("inf")), INV), (dict(rep=float("nan")), INV),
    (dict(freq=float("nan")), INV), (dict(pres=float("inf")), INV), (dict(cs=99), INV), (dict(cs=-1), INV), (dict(bs=1), INV),
    (dict(als=3), INV), (dict(x=P[0] + 2), ALIGN), (dict(counts=P[1] + 1), ALIGN), (dict(al=P[5] + 2), ALIGN),
    (dict(out=P[6] + 1), ALIGN), (dict(am=P[7] + 2), ALIGN), (dict(bias=P[4] + 2), ALIGN), (dict(tok=P[3] + 2), ALIGN),
    (dict(ws=None), WS), (dict(ws=P[8] + 4), WS), (dict(ws_bytes=16), WS)])
def test_adjust_refusals(lib, bad, status):
    assert call(lib.nt_logits_adjust, ADJUST, **bad) == status


LAYOUT = dict(parent=P[0], B=40, pos0=0, mask=P[1], words=2, pos=P[2], n_bad=None, stream=None)
ACCEPT = dict(parent=P[0], token=P[1], argmax=P[2], B=9, emit=P[3], path=P[4], n=P[5], stream=None)
COUNTS = dict(tokens=P[0], index=None, n=5, n_dev=None, V=100, counts=P[1], n_bad=None, stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(parent=None), INV), (dict(mask=None), INV), (dict(B=0), INV), (dict(B=257, words=9), INV), (dict(words=1), INV),
    (dict(pos0=2 ** 31 - 1), INV), (dict(parent=P[0] + 1), ALIGN), (dict(pos=P[2] + 2), ALIGN)])
def test_layout_refusals(lib, bad, status):
    assert call(lib.nt_tree_layout, LAYOUT, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(parent=None), INV), (dict(token=None), INV), (dict(argmax=None), INV), (dict(emit=None), INV), (dict(path=None), INV),
    (dict(n=None), INV), (dict(B=0), INV), (dict(B=257), INV), (dict(token=P[1] + 2), ALIGN), (dict(n=P[5] + 1), ALIGN)])
def test_accept_refusals(lib, bad, status):
    assert call(lib.nt_tree_accept, ACCEPT, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=None), INV), (dict(counts=None), INV), (dict(n=-1), INV), (dict(V=0), INV), (dict(tokens=P[0] + 2), ALIGN),
    (dict(index=P[2] + 1), ALIGN), (dict(counts=P[1] + 2), ALIGN)])
def test_counts_refusals(lib, bad, status):
    assert call(lib.nt_token_counts, COUNTS, **bad) == status


def commit_args(k=(P[0], P[1]), v=(P[2], P[3])):
    arr = lambda a: (ctypes.c_void_p * len(a))(*a)  # noqa: E731
    return dict(k=arr(k), v=arr(v), L=len(k), Hkv=2, D=128, ts=64, path=P[4], n=P[5], B=8, src=40, dst=32, stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(L=0), INV), (dict(Hkv=0), INV), (dict(Hkv=65536), INV), (dict(D=100), UNSUP),
    (dict(D=512), UNSUP), (dict(B=0), INV), (dict(B=257), INV), (dict(path=None), INV), (dict(n=None), INV), (dict(src=57), INV),
    (dict(dst=-1), INV), (dict(dst=41), INV), (dict(path=P[4] + 2), ALIGN)])
def test_commit_refusals(lib, bad, status):
    assert call(lib.nt_tree_commit, commit_args(), **bad) == status
    assert call(lib.nt_tree_commit, commit_args(k=(P[0], 0))) == INV
    assert call(lib.nt_tree_commit, commit_args(v=(P[2], P[3] + 8))) == ALIGN


def test_binding_refuses_what_the_abi_cannot_see(lib):
    f32, bf = torch.float32, torch.bfloat16
    q, k = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64)
    c = torch.zeros(2, 16, 64, dtype=bf)
    good = [q, k, k, None, None, 1e-6, None, 0, 1.0, torch.zeros(2, 4, 64), c, c]

    def append(**bad):
        names = ("q", "k", "v", "qg", "kg", "eps", "f", "layout", "amp", "q_out", "kc", "vc")
        nt.nt_qk_norm_rope_append(*[bad.get(n, g) for n, g in zip(names, good)], pos=bad.get("pos"), stream=0)

    for bad in (dict(q=q.half()), dict(k=k.to(bf)), dict(q=torch.zeros(2, 64, 4).transpose(1, 2)), dict(k=torch.zeros(3, 2, 64)),
                dict(kc=c.float()), dict(vc=c[:, ::2]), dict(q_out=torch.zeros(2, 4, 64, dtype=bf)), dict(qg=torch.zeros(32)),
                dict(f=torch.zeros(16, dtype=f32)), dict(pos=torch.zeros(2, dtype=torch.int64)), dict(q=q[0])):
        with pytest.raises(nt.NtError) as e:
            append(**bad)
        assert e.value.status == INV, bad
    mask, ws = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    for bad in (dict(q=q.half()), dict(q=q.transpose(0, 1)), dict(k=c.float()), dict(mask=mask.long()), dict(mask=mask[:1]),
                dict(out=q.to(bf))):
        a = dict(q=q, k=c, v=c, prefix=4, row0=4, mask=mask, out=q, ws=ws)
        a.update(bad)
        with pytest.raises(nt.NtError) as e:
            nt.nt_tree_attention(*a.values(), stream=0)
        assert e.value.status == INV
    x, am = torch.zeros(3, 40), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(counts=torch.zeros(40)), dict(counts=torch.zeros(2, 40, dtype=torch.int32)), dict(bias=torch.zeros(39)),
                dict(allowed=torch.zeros(3, 1, dtype=torch.int32)), dict(argmax=am.long()), dict(out=torch.zeros(3, 41))):
        with pytest.raises(nt.NtError) as e:
            nt.nt_logits_adjust(x, **{**dict(argmax=am, ws=ws), **bad}, stream=0)
        assert e.value.status == INV
    with pytest.raises(nt.NtError):
        nt.pointer_array([c, c.float()])
    with pytest.raises(nt.NtError):
        nt.nt_tree_commit(nt.pointer_array([c]), nt.pointer_array([c, c]), 2, 64, 16, am, am, 4, 4, stream=0)


def test_plain_forms_against_closed_forms():
    rs = np.random.RandomState(0)
    # a chain's ancestors are the lower triangle; a star's are itself and the root
    assert np.array_equal(_tree.ancestors(_tree.parents(rs, 5, "chain")), np.tril(np.ones((5, 5), bool)))
    star = np.eye(4, dtype=bool)
    star[:, 0] = True
    assert np.array_equal(_tree.ancestors(_tree.parents(rs, 4, "star")), star)
    # equal scores average the visible values
    v = rs.randn(1, 6, 2)
    out = _tree.attend(np.zeros((2, 1, 2)), rs.randn(1, 6, 2), v, 3, 4, np.array([[1, 0], [0, 0]], bool))
    assert np.allclose(out[0, 0], v[0, [0, 1, 2, 4]].mean(0)) and np.allclose(out[1, 0], v[0, :3].mean(0))
    # a quarter turn swaps a pair
    y = _tree.rotate(np.array([[[1.0, 0.0, 5.0]]]), None, 0.0, np.array([np.pi / 2]), 1, 1.0, np.array([1]))
    assert np.allclose(y[0, 0], [0.0, 1.0, 5.0])
    y = _tree.adjust(np.array([[2.0, -2.0, 1.0]]), np.array([[1, 2, 0]]), 2.0, 0.5, 0.25, None, None)
    assert np.allclose(y, [[0.25, -5.25, 1.0]])
    assert _tree.accept([-1, 0, 0, 1], [9, 5, 5, 7], [5, 7, 3, 8]) == ([0, 1, 3], [5, 7, 8])


def test_attention_plan_covers_every_tile(tmp_path):
    """tests/host/tree_plan_check.cu: the split of the attention's work over CTAs, host functions only."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "tree_plan_check")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O2", "-I",
                        os.path.join(root, "packed_weight_gemv_gb300", "csrc"), os.path.join(root, "tests", "host", "tree_plan_check.cu"),
                        "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr
