"""The package on a torch without CUDA: imports, builds tables, refuses tensors."""
import os
import subprocess
import sys

WITHOUT = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import lossless_diffusion_speculative_b200 as lib
turns, magnitude = lib.orthrus_rope_table(64, 1e4)
assert turns.numel() == 32 and magnitude == 1.0
x = torch.zeros(2, 64)
try:
    lib.orthrus_rmsnorm(x, x[0], 1e-6, out=x)
except ValueError:
    print("imported")
"""


def test_package_imports_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
