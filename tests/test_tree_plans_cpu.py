"""How the tree-verify kernels split their work over CTAs: host arithmetic of the library, compiled and run here."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# (rows of a group, B, V): logits whose rows the adjustments walk in groups, on a GPU of 152 SMs; tests/test_gpu_tree_range.py
# runs them
GROUPED_ROWS = [(8, 64, 151936), (16, 128, 151936), (9, 67, 151935), (7, 200, 40004), (7, 131, 60001), (13, 97, 300007),
                (5, 33, 151936)]


def compiled(name, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / name)
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O2", "-I",
                        os.path.join(ROOT, "packed_weight_gemv_gb300", "csrc"), os.path.join(ROOT, "tests", "host", name + ".cu"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return lambda *args: subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=120)


def test_adjustments_cover_every_row(tmp_path):
    run = compiled("adjust_plan_check", tmp_path)
    r = run()
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr
    got = [int(x) for x in run(*[n for _, B, V in GROUPED_ROWS for n in (B, V)]).stdout.split()]
    assert got == [g for g, _, _ in GROUPED_ROWS]


def test_attention_plans_with_clusters(tmp_path):
    r = compiled("tree_cluster_check", tmp_path)()
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr
