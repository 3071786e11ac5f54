"""Rules that the sources of the paged-cache kernels keep so that launches that overlap are safe, checked by reading; and how their
work is cut over CTAs, compiled from the library's header and run on the host."""
import os
import re
import shutil
import subprocess

import pytest

from packed_weight_gemv_gb300 import build as nt_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "packed_weight_gemv_gb300", "csrc")
NEW = ["nt_pages.cu", "nt_pages.cuh", "nt_beam.cu", "nt_paged.cuh", "nt_paged_few.cu", "nt_paged_many.cu", "nt_paged_attention.cu"]


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_tensor_memory_is_allocated_before_the_next_launch_begins():
    text = code("nt_paged_many.cu")
    kernel = text[text.index("paged_many_kernel"):text.index("paged_join_kernel")]
    at = kernel.index("tm_alloc(")
    begin = re.search(r"dependent_launch_wait\(\)|dependent_launch_begin\(\)", kernel).start()
    assert at < kernel.index("__syncthreads();", at) < begin
    assert kernel.count("tm_alloc(") == kernel.count("tm_free(") == 1


@pytest.mark.parametrize("name", NEW)
def test_inputs_that_the_kernel_before_writes_are_not_promised_constant(name):
    text = code(name)
    assert "__ldg(" not in text and "ld.global.nc" not in text
    assert not re.search(r"const\s+[\w:]+\s*\*\s*__restrict__", text)


@pytest.mark.parametrize("name", [n for n in NEW if n.endswith(".cu") and n != "nt_paged_attention.cu"])
def test_every_kernel_waits_for_the_one_before(name):
    text = code(name)
    kernels = [m.start() for m in re.finditer(r"__global__", text)]
    assert kernels
    for a, b in zip(kernels, kernels[1:] + [len(text)]):
        assert text[a:b].count("dependent_launch_wait();") == 1


def test_the_cut_of_the_work(tmp_path):
    """Random units over random grids: every tile is in one piece, the parts of a unit are those of the CTAs the join asks for, and no CTA
    leaves two parts in one place."""
    exe = tmp_path / "cut"
    cmd = [nt_build.nvcc(), *nt_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-o", str(exe),
           os.path.join(ROOT, "tests", "host", "paged_cut_check.cu")]
    if not shutil.which(cmd[0]):
        pytest.skip("no nvcc")
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert "ok" in r.stdout
