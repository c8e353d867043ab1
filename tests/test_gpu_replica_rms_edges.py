"""The replica's RMS norm at its edges, on the GPU: empty batches with their
workspace. Helpers as in test_gpu_replica_rms.py."""
import pytest

from test_gpu_replica_ops import torch, v  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rms_of_no_rows_with_its_workspace(torch, v):  # noqa: F811
    """As a caller has it: the query, the scratch, the call."""
    for rows, cols in ((0, 4096), (0, 50000), (5, 0), (0, 0)):
        ws = torch.empty(v.vrcclRmsNormWorkspace(rows, cols), device="cuda", dtype=torch.uint8)
        x, dg = torch.empty(rows, cols, device="cuda"), torch.ones(cols, device="cuda")
        rstd = torch.empty(rows, device="cuda")
        v.vrcclRmsNormForward(x, None, None, None, x, rstd, rows, cols, "float32", "float32")
        v.vrcclRmsNormBackward(x, None, x, None, rstd, x, dg, rows, cols, "float32", "float32", ws, ws.numel())
        assert (dg == 0).all()
