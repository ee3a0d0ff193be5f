"""The package imports where PyTorch is built without CUDA: what such a build lacks is looked up in calls."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import rank_gradient_sketching_philox_gb300 as rgs
from rank_gradient_sketching_philox_gb300 import binding, dataparallel, diagnostics, optimizer, policy_sync, train_example
assert rgs.code_rows(3, 20, device="cpu").stride() == (32, 1)
for call in (lambda: rgs.rms_norm_forward(torch.zeros(4, 16), None, Y=torch.zeros(4, 16)),
             lambda: rgs.quantize_blocks(torch.zeros(4, 16), rgs.code_rows(4, 16, device="cpu"), torch.zeros(4, 1)),
             lambda: rgs.grad_problems([torch.zeros(4)])):
    try:
        call()
    except ValueError:
        continue
    raise AssertionError("tensors of the CPU were taken")
"""


def test_the_package_imports_without_pytorchs_cuda_functions():
    p = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
