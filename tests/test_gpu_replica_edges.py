"""The operators of a replica at the edges of what they take: short rows on
every skew, extreme values, operands side by side, strides past 2^31 bytes.
Helpers, definitions and tolerances as in test_gpu_replica_ops.py."""
import numpy as np
import pytest

from oracle import replica as o
from test_gpu_replica_ops import EPS, FLOATS, TINY, U, Mat, _close, _host, _norm_check, _rng, torch, v  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ layer norm

@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 7, 9])
def test_norm_short_rows_on_every_skew(torch, v, cols, dtype):  # noqa: F811
    """Rows of a few elements share 16-byte blocks with the matrix's ends."""
    for rows in (1, 2, 3, 9, 400):
        for pad, offset in ((0, 0), (0, 1), (1, 3), (2, 6), (0, 7)):
            _norm_check(torch, v, rows, cols, dtype, "float32", pad, offset)


# ------------------------------------------------------------ status

def test_async_error_waits_for_every_stream(torch, v):  # noqa: F811
    """Work on a non-blocking stream is over when the query returns."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1)
    assert v.vrcclReplicaGetAsyncError() == 0  # the kernels' module is loaded, which waits too
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # a fifth of a second
    assert v.vrcclReplicaGetAsyncError() == 0
    assert side.query()
