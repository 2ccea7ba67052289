"""The package imports with a torch that was built without CUDA; what needs a GPU fails where it is called."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import speculative_decode_verify_w4a16_gb300 as sv
from speculative_decode_verify_w4a16_gb300 import verify_step
for call in (lambda: sv.quantize(torch.zeros(128, 128)),
             lambda: sv.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32))):
    try:
        call()
    except (ValueError, RuntimeError, AssertionError) as e:
        print("refused:", e)
    else:
        raise SystemExit("a CPU tensor was taken")
"""


def test_the_package_imports_without_cuda():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.count("refused:") == 2
