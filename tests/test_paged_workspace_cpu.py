"""Where the paged attention keeps what in its workspace, compiled from the library's header and run on the host."""
import os
import shutil
import subprocess

import pytest

from packed_weight_gemv_gb300 import build as nt_build
from packed_weight_gemv_gb300 import nt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "packed_weight_gemv_gb300", "csrc")


def test_counters_stand_where_no_other_call_writes(tmp_path):
    exe = tmp_path / "workspace"
    cmd = [nt_build.nvcc(), *nt_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-o", str(exe),
           os.path.join(ROOT, "tests", "host", "paged_workspace_check.cu")]
    if not shutil.which(cmd[0]):
        pytest.skip("no nvcc")
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert "ok" in r.stdout


def test_the_largest_call_sizes_the_workspace():
    """One workspace for every step of a server: that of the most tokens; sequences do not enter."""
    for Hq, Hkv, D in ((32, 8, 128), (32, 32, 64), (64, 1, 128)):
        sizes = [nt.nt_paged_attention_workspace_size(T, min(T, 4096), Hq, Hkv, D) for T in (1, 2, 8, 9, 100, 130, 1000, 5000)]
        assert sizes == sorted(sizes)
        assert len({nt.nt_paged_attention_workspace_size(60, S, Hq, Hkv, D) for S in (1, 17, 60)}) == 1
