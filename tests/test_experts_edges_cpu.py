"""Host-side tests of the operators around the experts at the edges: rules of the host, and what needs no GPU."""
import os
import subprocess
import sys

import pytest

from tp_reduce_residual_gb300 import experts


@pytest.mark.parametrize("n,M,K,taken", [
    (4096, 32768, 5120, True), (6000, 24000, 4096, True), (2048, 20480, 8192, True), (2048, 16384, 1024, True), (300, 31000, 544, True),
    (2048, 8192, 8192, False), (1000, 9999, 8192, False), (1000, 10000, 8192, True),      # 9000 places more than rows
    (4096, 16384, 1024, False), (4096, 16384, 2048, True),                                # below 2^25, 8 places a row
    (16384, 65532, 2048, False), (16384, 65536, 2048, True), (300, 30000, 544, False), (1, 2 ** 31 - 1024, 1 << 20, True)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_workspace_where_it_pays(n, M, K, taken, fmt):
    """Repeated rows go through the workspace where there are enough repeats and enough work for it."""
    assert (experts.quantize_workspace_bytes(n, M, K, fmt) > 0) == taken


def test_package_imports_without_cuda_in_torch():
    """Inputs, refusals and the build are there under a PyTorch that was built without CUDA."""
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "import tp_reduce_residual_gb300.experts\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
