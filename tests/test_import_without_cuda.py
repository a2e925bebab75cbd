"""The package without torch's private CUDA functions, as a torch built without CUDA has none (no
GPU): it imports, and calls refuse their arguments as ever."""
import os
import subprocess
import sys

CODE = r"""
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import qwen3_vl_decoder_b200 as q3
c = q3.config(2560, 32, 8, 9728)
try:
    q3.add_rms_norm_q8(c, torch.zeros(2, 2560, dtype=torch.bfloat16), None)
except q3.Q3VLError as e:
    print("refused:", e)
calls = []
class Fake:                       # what the fallbacks ask of torch.cuda
    cuda_stream = 1234
torch.cuda.is_initialized = lambda: True
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda d=None: calls.append(d) or Fake
assert q3._stream().value == 1234 and calls == [3], calls
print("streams")
"""


def test_import_and_refusals_without_torchs_private_functions():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, cwd=root,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-1500:]
    assert "refused:" in r.stdout and "streams" in r.stdout
