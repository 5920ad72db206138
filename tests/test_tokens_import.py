"""The package's planning and host helpers import with any torch, also one built
without GPU support.  No GPU work."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# What a torch without GPU support lacks.
CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    delattr(torch._C, name)
import gradient_reduce_zero_amd as grz
assert grz.plan_buckets([100, 200])
try:
    grz.dp_embed_lookup(torch.zeros(2, 2), torch.zeros(2, dtype=torch.long), torch.zeros(2, 2))
except ValueError as e:
    print("refused:", e)
"""


def test_import_with_a_torch_without_gpu_support():
    res = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, cwd=ROOT)
    assert res.returncode == 0, res.stderr
    assert "refused: table must be on the GPU" in res.stdout
