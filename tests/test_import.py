"""The package's host side on a torch build without CUDA, which lacks the private functions of torch._C that
the calls use."""
import subprocess
import sys

CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import video_dit_dynamic_token_b200 as lx
from video_dit_dynamic_token_b200 import pipeline, ulysses
assert lx.lx_nvfp4_gemv_ws_size(9, 64, 320) > 0
assert lx.keep_count(16, 0.25) == 4
t = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
cu = torch.tensor([0, 8], dtype=torch.int32)
try:
    lx.lx_attn_packed(t, t, t, cu, cu)
except ValueError as e:
    assert "CUDA tensors" in str(e)
else:
    raise AssertionError("CPU tensors were taken")
"""


def test_imports_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
