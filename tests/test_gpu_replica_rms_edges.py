"""The replica's RMS norm at its edges, on the GPU: empty batches with their
workspace, rows that are read twice, the widest that are held and the narrowest,
more of each than are at work at once. Helpers as in test_gpu_replica_rms.py."""
import pytest

from test_gpu_replica_ops import Mat, _rng, torch, v  # noqa: F401
from test_gpu_replica_rms import _backward, _forward

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


@pytest.mark.parametrize("rows,cols,dtype,pad", [(330, 16392, "bfloat16", 0), (330, 20001, "float32", 0), (620, 20001, "float16", 3), (330, 15001, "float32", 0)])
def test_rms_of_more_rows_read_twice_than_blocks(torch, v, rows, cols, dtype, pad):  # noqa: F811
    """A block goes on to another row, and sums several into a column of the weight's gradient."""
    _forward(torch, v, rows, cols, dtype, "float32", pad)
    _backward(torch, v, rows, cols, dtype, "float32", pad)
    _backward(torch, v, rows, cols, dtype, "float32", pad, dsum=False, affine=False)


@pytest.mark.parametrize("cols,dtype", [(16392, "bfloat16"), (20001, "bfloat16"), (20001, "float32"), (15001, "float32"), (16384, "float32")])
def test_rms_of_rows_read_twice_in_place(torch, v, cols, dtype):  # noqa: F811
    """dx in the place of each input: what a column's sum needs has been read."""
    g, rows = _rng(11), 330
    make = lambda q: Mat(torch, rows, cols, dtype, q)  # noqa: E731
    a = [torch.as_tensor(g.standard_normal((rows, cols))) for _ in range(3)]
    rstd = torch.rand(rows, device="cuda")
    ws = torch.empty(v.vrcclRmsNormWorkspace(rows, cols), device="cuda", dtype=torch.uint8)
    want, dg, dg2 = make(None), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")

    def back(dy, ds, s, dx, grad):
        v.vrcclRmsNormBackward(dy.ptr, ds.ptr, s.ptr, None, rstd, dx.ptr, grad, rows, cols, dtype, "float32", ws, ws.numel())

    back(*[make(q) for q in a], want, dg)
    for over in range(3):
        m = [make(q) for q in a]
        back(*m, m[over], dg2)
        assert torch.equal(m[over].view, want.view) and torch.equal(dg, dg2) and m[over].intact()


@pytest.mark.parametrize("rows,cols,dtype", [(900, 16384, "bfloat16"), (700, 13000, "float16"), (700, 12800, "float32")])
def test_rms_of_many_wide_rows_on_boundaries(torch, v, rows, cols, dtype):  # noqa: F811
    """Teams of a whole block, whose stages are filled again."""
    _forward(torch, v, rows, cols, dtype, "float32")
    _forward(torch, v, rows, cols, dtype, "float32", residual=False, quant="e4m3", group=128, with_y=False)
    _backward(torch, v, rows, cols, dtype, "float32")


@pytest.mark.parametrize("rows,cols,dtype", [(160001, 24, "bfloat16"), (90001, 64, "float32"), (90003, 128, "bfloat16"), (50002, 120, "float16")])
def test_rms_of_more_narrow_rows_than_are_at_work(torch, v, rows, cols, dtype):  # noqa: F811
    _forward(torch, v, rows, cols, dtype, "float32")
    _forward(torch, v, rows, cols, dtype, dtype, residual=False, quant="int8", group=32, with_y=False)
    _backward(torch, v, rows, cols, dtype, "float32")


def test_rms_of_rows_whose_squares_leave_the_range(torch, v):  # noqa: F811
    """As the header says: an inverse root of 0 where the sum of squares passes binary32, infinite where it is 0 and eps too."""
    for rows, cols in ((5, 64), (5, 1001), (3, 20001)):
        x, y, rstd = torch.ones(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda"), torch.empty(rows, device="cuda")
        x[0], x[1] = 1e20, 0
        v.vrcclRmsNormForward(x, None, None, None, y, rstd, rows, cols, "float32", "float32", 0.0)
        assert rstd[0] == 0 and (y[0] == 0).all() and rstd[1] == float("inf") and (rstd[2:] == 1).all() and (y[2:] == 1).all()
