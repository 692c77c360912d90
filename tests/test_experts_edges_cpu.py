"""Host-side tests of the operators around the experts at the edges: what needs no GPU stays without one."""
import os
import subprocess
import sys


def test_package_imports_without_cuda_in_torch():
    """Inputs, refusals and the build are there under a PyTorch that was built without CUDA."""
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "import tp_reduce_residual_gb300.experts\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
