"""The package needs torch's public interface only: it can be imported with a torch
that was built without a GPU backend."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import mxfp4_routed_expert_router_amd as moe
assert moe.moe_fp4_linear_workspace_size(64, 512, 512) >= 0
print("imported")
"""


def test_import_without_a_gpu_backend():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
