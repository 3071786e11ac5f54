"""Rules that the kernels' sources keep so that launches that overlap (programmatic dependent launches) are safe. They are
checked by reading: what they prevent, a wait without end or a stale read, is nothing to provoke on a GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_weight_gemv_gb300", "csrc")
BEGINS = re.compile(r"dependent_launch_wait\(\)|dependent_launch_begin\(\)|griddepcontrol\.launch_dependents")
ALLOCATES = "tcgen05.alloc."


def code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def functions(text):
    """The pieces of a source between lines that begin a function or a template at the margin."""
    at = [m.start() for m in re.finditer(r"^(?:template|__global__|__device__|static|inline)\b", text, re.M)] + [len(text)]
    return [text[a:b] for a, b in zip(at, at[1:])]


def allocating():
    return [(os.path.basename(p), f) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) for f in functions(code(p)) if ALLOCATES in f]


def test_the_kernels_that_allocate_are_found():
    assert {n for n, _ in allocating()} == {"nt_gemm_tc.cu", "nt_gemv_tc8.cu", "nt_tree_attention.cu", "nt_tree_few.cu"}


@pytest.mark.parametrize("name,text", allocating(), ids=[n for n, _ in allocating()])
def test_tensor_memory_is_allocated_before_the_next_launch_begins(name, text):
    """Otherwise a CTA of the next kernel may hold an SM's tensor memory while it waits for this grid, and a CTA of this grid
    wait for that memory."""
    at = text.index(ALLOCATES)
    assert not BEGINS.search(text[:at]), f"{name} lets the next launch begin before it has its tensor memory"
    begin = BEGINS.search(text, at)
    assert begin is None or "__syncthreads();" in text[at:begin.start()], f"{name}: other threads may let the next launch begin earlier"


@pytest.mark.parametrize("name", ["nt_tree.cu", "nt_tree.cuh", "nt_tree_attention.cu", "nt_tree_attn.cuh", "nt_tree_few.cu",
                                  "nt_logits_adjust.cu", "nt_qk_rope.cu"])
def test_inputs_that_the_kernel_before_writes_are_not_promised_constant(name):
    """These kernels become resident while the one before still writes their inputs: a load that the language lets the compiler
    move, or cache for the kernel's lifetime, could return the old data."""
    text = code(os.path.join(CSRC, name))
    assert "__ldg(" not in text and "ld.global.nc" not in text
    assert not re.search(r"const\s+[\w:]+\s*\*\s*__restrict__", text)
