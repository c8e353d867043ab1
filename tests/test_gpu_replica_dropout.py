"""The replica's dropout on the GPU against its definition (oracle/replica.py):
the mask bit for bit, values to one rounding, strides, alignment, in place,
splits over calls, streams and graphs. Helpers and U, EPS, TINY as in
test_gpu_replica_ops.py."""
import numpy as np
import pytest

from oracle import replica as o
from test_gpu_replica_ops import EPS, FLOATS, TINY, U, Mat, _close, _rng, torch, v  # noqa: F401

pytestmark = pytest.mark.gpu

SEED = 0x9E3779B97F4A7C15


def _seed(torch, value=SEED):  # noqa: F811
    return torch.tensor([value - (1 << 64) if value >> 63 else value], device="cuda", dtype=torch.int64)


def _check(torch, v, rows, cols, dtype, p, pad=0, offset=0, residual=True, yskew=None, number=5, first=0):  # noqa: F811
    g = _rng(rows * 1000 + cols)
    x = Mat(torch, rows, cols, dtype, g.standard_normal((rows, cols)), pad, offset)
    r = Mat(torch, rows, cols, dtype, g.standard_normal((rows, cols)), pad, offset) if residual else None
    y = Mat(torch, rows, cols, dtype, None, pad, offset if yskew is None else yskew)
    seed = _seed(torch)
    kept, scale = o.dropout_mask(rows, cols, p, SEED, number, first)
    X, R = x.get(), r.get() if residual else np.zeros((rows, cols))
    v.vrcclDropoutForward(x.ptr, r.ptr if residual else None, y.ptr, rows, cols, dtype, p, seed, number, first, ldx=x.ld,
                          ldr=r.ld if residual else None, ldy=y.ld)
    want = np.where(kept, X * scale, 0) + R
    # the scale is rounded once, the product added (or rounded) once in binary32, the result to its type
    tol = U[dtype] * 1.01 * np.abs(want) + 2 * EPS * (np.abs(X) * scale + np.abs(R)) + TINY[dtype]
    _close(y.get(), want, tol, "y")
    if not residual:
        assert np.array_equal(y.get() != 0, kept & (X != 0))
    assert y.intact() and x.intact()
    dx = Mat(torch, rows, cols, dtype, None, pad, offset if yskew is None else yskew)
    v.vrcclDropoutBackward(x.ptr, dx.ptr, rows, cols, dtype, p, seed, number, first, lddy=x.ld, lddx=dx.ld)
    want = np.where(kept, X * scale, 0)
    _close(dx.get(), want, U[dtype] * 1.01 * np.abs(want) + 2 * EPS * np.abs(want) + TINY[dtype], "dx")
    assert dx.intact()


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (1, 7, 0, 1), (3, 8, 0, 0), (5, 9, 0, 0), (4, 64, 0, 0),
                                                  (4, 64, 8, 0), (7, 257, 0, 0), (6, 255, 1, 3), (3, 520, 0, 1), (2, 1001, 6, 0),
                                                  (9, 100, 4, 4), (3, 1024, 0, 8)])
def test_dropout(torch, v, rows, cols, pad, offset, dtype):  # noqa: F811
    _check(torch, v, rows, cols, dtype, 0.25, pad, offset)
    _check(torch, v, rows, cols, dtype, 0.1, pad, offset, residual=False, number=1 << 40, first=(1 << 33) + 5)


@pytest.mark.parametrize("rows,cols,pad,offset", [(70, 3, 0, 0), (33, 65, 0, 0), (17, 127, 0, 2), (5, 250, 3, 0), (6, 1001, 0, 0), (5, 4097, 0, 1),
                                                  (4, 2048, 3, 0)])
def test_dropout_of_odd_rows(torch, v, rows, cols, pad, offset):  # noqa: F811
    """Several rows a warp, and warps inside a row that look at the next one's beginning."""
    for dtype in ("float32", "float16"):
        _check(torch, v, rows, cols, dtype, 0.3, pad, offset)
        _check(torch, v, rows, cols, dtype, 0.3, pad, offset, residual=False, yskew=(offset + 3) % 8)


def test_dropout_counters_past_32_bits(torch, v):  # noqa: F811
    """Row numbers at which a block's counters, and a warp's, pass a multiple of 2^32."""
    for rows, cols, pad in ((100, 64, 0), (100, 64, 8), (9, 1001, 0)):
        per = -(-cols // 8)
        for upper in (1, 5):
            _check(torch, v, rows, cols, "bfloat16", 0.5, pad, first=(upper << 32) // per - 5)


@pytest.mark.parametrize("skew", range(8))
def test_dropout_output_on_every_skew(torch, v, skew):  # noqa: F811
    _check(torch, v, 3, 300, "bfloat16", 0.5, 3, 2, yskew=skew)
    _check(torch, v, 3, 261, "float32", 0.5, 0, 1, yskew=skew)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 2.0 ** -16, 0.5, 1 - 2.0 ** -16, 1.0])
def test_dropout_probabilities(torch, v, p):  # noqa: F811
    for rows, cols, pad in ((3, 64, 0), (2, 77, 1)):
        _check(torch, v, rows, cols, "float32", p, pad, residual=True)
        _check(torch, v, rows, cols, "bfloat16", p, pad, residual=False)


def test_dropout_of_many_rows_matches_its_parts(torch, v):  # noqa: F811
    """A large call (four chunks a thread) has the mask of its pieces, on any stride; each piece the oracle's."""
    rows, cols = 5000, 776
    seed = _seed(torch)
    x = torch.ones(rows, cols, device="cuda", dtype=torch.bfloat16)
    y, odd = torch.empty_like(x), torch.empty(rows, cols + 3, device="cuda", dtype=torch.bfloat16)[:, :cols]
    v.vrcclDropoutForward(x, None, y, rows, cols, "bfloat16", 0.3, seed, 9)
    v.vrcclDropoutForward(x, None, odd, rows, cols, "bfloat16", 0.3, seed, 9)
    assert torch.equal(y, odd)
    gaps = torch.empty(rows, cols + 8, device="cuda", dtype=torch.bfloat16)[:, :cols]
    v.vrcclDropoutForward(x, None, gaps, rows, cols, "bfloat16", 0.3, seed, 9)
    assert torch.equal(y, gaps)
    wide = torch.ones(rows, cols + 8, device="cuda", dtype=torch.bfloat16)[:, :cols]
    gaps.zero_()
    v.vrcclDropoutForward(wide, None, gaps, rows, cols, "bfloat16", 0.3, seed, 9)
    assert torch.equal(y, gaps)
    part = torch.empty(13, cols, device="cuda", dtype=torch.bfloat16)
    for at in (0, 1, 2500, rows - 13):
        v.vrcclDropoutForward(x[at:at + 13], None, part, 13, cols, "bfloat16", 0.3, seed, 9, at)
        assert torch.equal(part, y[at:at + 13])
        kept, _ = o.dropout_mask(13, cols, 0.3, SEED, 9, at)
        assert np.array_equal((part != 0).cpu().numpy(), kept)
    share = (y != 0).double().mean().item()
    assert abs(share - (1 - round(0.3 * 65536) / 65536)) < 6 * (0.3 * 0.7 / (rows * cols)) ** 0.5


def test_dropped_elements_may_hold_anything(torch, v):  # noqa: F811
    kept, scale = o.dropout_mask(4, 96, 0.5, SEED, 0, 0)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.full((4, 96), bad, device="cuda")
        x[torch.as_tensor(kept).cuda()] = 2.0
        y = torch.empty_like(x)
        for p_res in (None, torch.ones_like(x)):
            v.vrcclDropoutForward(x, p_res, y, 4, 96, "float32", 0.5, _seed(torch))
            want = np.where(kept, 2 * scale, 0) + (p_res is not None)
            assert np.array_equal(y.cpu().numpy(), want.astype(np.float32))


@pytest.mark.parametrize("cols,pad", [(128, 0), (131, 0), (131, 5), (1001, 0), (4001, 6)])
def test_dropout_in_place(torch, v, cols, pad):  # noqa: F811
    g = _rng(3)
    a, b = g.standard_normal((40, cols)), g.standard_normal((40, cols))
    want = Mat(torch, 40, cols, "bfloat16", None, pad)
    x, r = Mat(torch, 40, cols, "bfloat16", a, pad), Mat(torch, 40, cols, "bfloat16", b, pad)
    args = (40, cols, "bfloat16", 0.2, _seed(torch), 3, 4)
    v.vrcclDropoutForward(x.ptr, r.ptr, want.ptr, *args, ldx=x.ld, ldr=r.ld, ldy=want.ld)
    for over in (x, r):
        keep = over.buf.clone()
        v.vrcclDropoutForward(x.ptr, r.ptr, over.ptr, *args, ldx=x.ld, ldr=r.ld, ldy=over.ld)
        assert torch.equal(over.view, want.view) and over.intact()
        over.buf.copy_(keep)
    v.vrcclDropoutBackward(x.ptr, want.ptr, *args, lddy=x.ld, lddx=want.ld)
    v.vrcclDropoutBackward(x.ptr, x.ptr, *args, lddy=x.ld, lddx=x.ld)
    assert torch.equal(x.view, want.view) and x.intact()


def test_dropout_seed_is_read_when_the_graph_runs(torch, v):  # noqa: F811
    """A captured step draws another mask once the seed changes, and the same one while it does not; two graphs share nothing."""
    seed, x = _seed(torch, 1), torch.ones(64, 520, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    v.vrcclDropoutForward(x, None, y, 64, 520, "float32", 0.4, seed, 2)
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for out in (y, z):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                v.vrcclDropoutForward(x, None, out, 64, 520, "float32", 0.4, seed, 2)
            graphs.append(graph)
    for value in (7, 7, 8, (1 << 63) + 1):
        seed.copy_(_seed(torch, value))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        kept, _ = o.dropout_mask(64, 520, 0.4, value, 2, 0)
        assert np.array_equal((y != 0).cpu().numpy(), kept) and torch.equal(y, z)


def test_dropout_on_another_stream(torch, v):  # noqa: F811
    x, y, seed = torch.ones(100, 512, device="cuda"), torch.zeros(100, 512, device="cuda"), _seed(torch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.mul_(3)
    v.vrcclDropoutForward(x, None, y, 100, 512, "float32", 0.5, seed, stream=side)
    side.synchronize()
    kept, _ = o.dropout_mask(100, 512, 0.5, SEED, 0, 0)
    assert np.array_equal(y.cpu().numpy(), np.where(kept, 6.0, 0).astype(np.float32))


def test_dropout_rows_beyond_32_bits(torch, v):  # noqa: F811
    """Rows more than 2^32 elements apart."""
    ld = (1 << 31) + 64
    x = torch.empty(2 * ld + 200, device="cuda", dtype=torch.bfloat16)
    view = x.as_strided((3, 200), (ld, 1))
    y = torch.empty(3, 200, device="cuda", dtype=torch.bfloat16)
    for shift in (0, 1):
        rows = x.as_strided((3, 199), (ld, 1), shift) if shift else view
        rows.fill_(1)
        n = rows.shape[1]
        v.vrcclDropoutForward(rows, None, y, 3, n, "bfloat16", 0.5, _seed(torch), ldy=200)
        v.vrcclDropoutBackward(rows, rows, 3, n, "bfloat16", 0.5, _seed(torch))
        assert torch.equal(rows, y[:, :n])
        kept, _ = o.dropout_mask(3, n, 0.5, SEED, 0, 0)
        assert np.array_equal((y[:, :n] != 0).cpu().numpy(), kept)
