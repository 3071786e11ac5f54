"""The workspace size of nt_attention_decode is that of the device, even where it is the first call of a process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
from packed_weight_gemv_gb300 import nt
ws = torch.zeros(nt.nt_attention_workspace_size(1, 8, 1, 8000), dtype=torch.uint8, device="cuda")
q, k, v = torch.randn(1, 8, 128, device="cuda"), *(torch.randn(1, 8000, 128, device="cuda").bfloat16() for _ in range(2))
nt.nt_attention_decode(q, k, v, 1, 8, 1, 128, 8000, 8000, torch.empty_like(q), ws)
torch.cuda.synchronize()
print("ok")
"""


def test_size_before_any_other_call():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]
