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


# ------------------------------------------------------------ linear layer

@pytest.mark.parametrize("rows,outs,ins", [(4096, 4096, 256), (2048, 1536, 64), (5000, 136, 136)])
def test_linear_tiles_in_a_row_give_the_same_bits(torch, v, rows, outs, ins):  # noqa: F811
    """Every lane of an epilogue reads finished products: many short tiles a
    block, again and again, against the first pass and against 64 bits."""
    g = torch.Generator("cuda").manual_seed(1)
    x, w = (torch.randn(n, ins, generator=g, device="cuda").bfloat16() for n in (rows, outs))
    y = torch.empty(rows, outs, device="cuda", dtype=torch.bfloat16)
    first = None
    for _ in range(20):
        y.fill_(float("nan"))
        v.vrcclLinearForward(x, w, None, None, y, None, rows, outs, ins, "bfloat16")
        first = y.clone() if first is None else first
        assert torch.equal(y, first)
    X, W = x.double(), w.double()
    want = X @ W.t()
    off = (y.double() - want).abs() - U["bfloat16"] * 1.01 * want.abs() - (ins + 16) * 2 * EPS * (X.abs() @ W.abs().t())
    assert off.max().item() <= 0
