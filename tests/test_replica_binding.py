"""The binding of the replica's operators, no GPU needed."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def v():
    pytest.importorskip("torch")
    from ring_allreduce_reduction_gb300 import build
    build.build()
    from ring_allreduce_reduction_gb300 import vrccl
    return vrccl


def test_imports_where_torch_has_no_cuda(v):
    """Host-side calls work with a torch that was built without CUDA (no raw stream to ask for)."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "from ring_allreduce_reduction_gb300 import vrccl as v\n"
            "assert v.vrcclLayerNormWorkspace(4, 64) > 0\n"
            "assert v.vrcclShardRange(100, 'float32', 4, 0)[1] > 0\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
