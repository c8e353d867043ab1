"""The operators of a replica at the edges of what they take: short rows on
every skew, extreme values, operands side by side, strides past 2^31 bytes.
Helpers, definitions and tolerances as in test_gpu_replica_ops.py."""
import numpy as np
import pytest

from oracle import replica as o
from test_gpu_replica_ops import (EPS, FLOATS, TINY, U, Mat, _close, _distill_check, _distill_inputs, _host, _norm_check,  # noqa: F401
                                  _rng, torch, v)  # noqa: F401

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


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_slope_of_large_arguments(torch, v, dtype, act):  # noqa: F811
    """Every finite z has a finite slope: 0 or 1 once it is large, however its
    powers overflow."""
    top = float(torch.finfo(getattr(torch, dtype)).max)
    z = np.array([s * m for m in (1.0, 9.0, 40.0, 3e3, 6e4, 1e9, 2e13, 1e15, 1e19, 3e19, 1e30, 3e38) if m <= top
                  for s in (1, -1)] + [top, -top])
    rows, n = 16, z.size
    Z = Mat(torch, rows, n, dtype, np.tile(z, (rows, 1)))
    dy = Mat(torch, rows, n, dtype, _rng(5).standard_normal((rows, n)))
    db = torch.empty(n, device="cuda", dtype=getattr(torch, dtype))
    ws = torch.empty(v.vrcclLinearWorkspace("backward", rows, n, 8, dtype, act), device="cuda", dtype=torch.uint8)
    v.vrcclLinearBackward(dy.ptr, Z.ptr, None, None, None, None, db, rows, n, 8, dtype, act, ws, ws.numel())
    z, D = Z.get()[0], dy.get()
    with np.errstate(over="ignore", invalid="ignore"):
        slope = np.where(z > 100, 1.0, np.where(z < -100, 0.0, o.slope(np.clip(z, -100, 100), act)))
    want = (D * slope).sum(0)
    # as in _linear_back, with arguments no larger than where the slope is still moving
    es = (32 * EPS * np.abs(D) * (1 + np.minimum(np.abs(z), 50))).sum(0)
    _close(_host(db), want, U[dtype] * np.abs(want) * 1.01 + es + (rows + 16) * EPS * np.abs(D * slope).sum(0) + TINY[dtype], "dbias")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_gelu_is_rounded_once(torch, v, dtype):  # noqa: F811
    """gelu and its slope to one rounding of the type, in the tail too.

    Phi(-x) = exp(-x^2/2) R(x): the exponent, of at most 26 binary digits
    here (|z| <= 6), is rounded twice (52 EPS of it, times log 2, 36); the two
    special functions, the reciprocal and the polynomial add some 28 EPS.
    The slope adds a product with the same density."""
    u, some = U[dtype], 64 * EPS
    grid = torch.linspace(-6, 6, 4001, dtype=torch.float64).to(getattr(torch, dtype)).unique()
    z = grid.double().numpy()
    n = z.size
    # Phi of either sign without cancellation, by its definition in 64 bits
    phi = 0.5 * torch.special.erfc(torch.as_tensor(-z / np.sqrt(2))).numpy()
    dense = z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    w = torch.zeros(n, 8, device="cuda", dtype=grid.dtype)
    w[:, 0] = grid.cuda()
    for rows in (1, 20, 300):
        x, y = torch.zeros(rows, 8, device="cuda", dtype=grid.dtype), torch.empty(rows, n, device="cuda", dtype=grid.dtype)
        x[:, 0] = 1
        ws = torch.empty(max(256, v.vrcclLinearWorkspace("forward", rows, n, 8, dtype, "gelu")), device="cuda", dtype=torch.uint8)
        v.vrcclLinearForward(x, w, None, None, y, None, rows, n, 8, dtype, "gelu", ws, ws.numel())
        want = np.tile(z * phi, (rows, 1))
        _close(_host(y), want, (u + some) * np.abs(want) + TINY[dtype] / 2, f"gelu, {rows} rows")
    db = torch.empty(n, device="cuda", dtype=grid.dtype)
    one = torch.ones(1, n, device="cuda", dtype=grid.dtype)
    ws = torch.empty(v.vrcclLinearWorkspace("backward", 1, n, 8, dtype, "gelu"), device="cuda", dtype=torch.uint8)
    v.vrcclLinearBackward(one, grid.cuda(), None, None, None, None, db, 1, n, 8, dtype, "gelu", ws, ws.numel())
    _close(_host(db), phi + dense, u * np.abs(phi + dense) + 2 * some * (phi + np.abs(dense)) + TINY[dtype] / 2, "slope")


# ------------------------------------------------------------ distillation

@pytest.mark.parametrize("ttype", FLOATS)
@pytest.mark.parametrize("vocab", [700, 70001])
def test_distill_nan_teacher_is_kept(torch, v, vocab, ttype):  # noqa: F811
    """A NaN among the teacher's logits makes the row's loss and its entries' gradients NaN, and nothing else."""
    s, t, idx = _distill_inputs(4, vocab, 6, 9)
    t[1, 2] = np.nan
    t[2, 0], idx[2, 0] = np.nan, -1  # (outside the vocabulary: not kept)
    with np.errstate(invalid="ignore"):
        loss, d = _distill_check(torch, v, s, t, idx, "float32", ttype)
    assert np.array_equal(np.isnan(loss), [False, True, False, False])
    assert np.array_equal(np.flatnonzero(np.isnan(d[1])), np.sort(idx[1])) and np.isfinite(d[[0, 2, 3]]).all()


# ------------------------------------------------------------ column slices of one buffer

class Slices:
    """Matrices of one dtype side by side in one buffer (`together`), or each
    at the same place of a buffer of its own."""

    def __init__(self, torch, rows, widths, dtype, gap, together):  # noqa: F811
        at, self.ld = {}, gap
        for name, n in widths.items():
            at[name] = (self.ld, n)
            self.ld += n + gap
        self.ld += (-self.ld) % 8 if gap % 8 == 0 else 0
        new = lambda: torch.full((rows, self.ld), Mat.CANARY, device="cuda", dtype=getattr(torch, dtype))  # noqa: E731
        one = new()
        self.bufs = [one] if together else []
        self.t, self.at = {}, at
        for name, (c, n) in at.items():
            buf = one if together else new()
            if not together:
                self.bufs.append(buf)
            self.t[name] = buf[:, c:c + n]

    def __getitem__(self, name):
        return self.t[name].data_ptr()

    def gaps_intact(self):
        bad = 0
        for buf in self.bufs:
            a = buf.clone()
            for c, n in self.at.values():
                a[:, c:c + n] = Mat.CANARY
            bad += (a != Mat.CANARY).sum().item()
        return bad == 0


@pytest.mark.parametrize("gap", [0, 8, 3])
@pytest.mark.parametrize("rows,cols", [(40, 264), (700, 64), (333, 1001), (5, 9000), (3, 33001)])
def test_norm_column_slices(torch, v, rows, cols, gap):  # noqa: F811
    got = []
    for together in (False, True):
        b = Slices(torch, rows, {"x": cols, "y": cols, "dy": cols, "dx": cols}, "bfloat16", gap, together)
        g = torch.Generator("cuda").manual_seed(3)
        for n in ("x", "dy"):
            b.t[n].copy_(torch.randn(rows, cols, generator=g, device="cuda"))
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        ws = torch.empty(v.vrcclLayerNormWorkspace(rows, cols), device="cuda", dtype=torch.uint8)
        v.vrcclLayerNormForward(b["x"], None, None, b["y"], mean, rstd, rows, cols, "bfloat16", "float32", ldx=b.ld, ldy=b.ld)
        v.vrcclLayerNormBackward(b["dy"], b["x"], None, mean, rstd, b["dx"], dg, db, rows, cols, "bfloat16", "float32", ws,
                                 ws.numel(), lddy=b.ld, ldx=b.ld, lddx=b.ld)
        assert b.gaps_intact()
        got.append([t.clone() for t in (*b.t.values(), mean, rstd, dg, db)])
    assert all(torch.equal(a, c) for a, c in zip(*got))


@pytest.mark.parametrize("gap", [0, 8, 3])
@pytest.mark.parametrize("rows,outs,ins", [(1, 72, 64), (7, 40, 136), (33, 130, 65), (300, 264, 72), (1500, 1000, 96)])
def test_linear_column_slices(torch, v, rows, outs, ins, gap):  # noqa: F811
    got = []
    for together in (False, True):
        b = Slices(torch, rows, {"x": ins, "z": outs, "y": outs, "r": outs, "dy": outs, "dx": ins}, "bfloat16", gap, together)
        g = torch.Generator("cuda").manual_seed(4)
        for n in ("x", "r", "dy"):
            b.t[n].copy_(torch.randn(b.t[n].shape, generator=g, device="cuda"))
        w = (torch.randn(outs, ins, generator=g, device="cuda") / 8).bfloat16()
        dw = torch.empty_like(w)
        ws = torch.empty(v.vrcclLinearWorkspace("backward", rows, outs, ins, "bfloat16", "silu"), device="cuda", dtype=torch.uint8)
        v.vrcclLinearForward(b["x"], w, None, b["r"], b["y"], b["z"], rows, outs, ins, "bfloat16", "silu", ws, ws.numel(),
                             ldx=b.ld, ldr=b.ld, ldy=b.ld, ldz=b.ld)
        v.vrcclLinearBackward(b["dy"], b["z"], b["x"], w, b["dx"], dw, None, rows, outs, ins, "bfloat16", "silu", ws,
                              ws.numel(), lddy=b.ld, ldz=b.ld, ldx=b.ld, lddx=b.ld)
        assert b.gaps_intact()
        got.append([t.clone() for t in (*b.t.values(), dw)])
    assert all(torch.equal(a, c) for a, c in zip(*got))


@pytest.mark.parametrize("gap", [0, 8, 3])
@pytest.mark.parametrize("rows,vocab", [(40, 1000), (3, 70001)])
def test_distill_column_slices(torch, v, rows, vocab, gap):  # noqa: F811
    got = []
    _, t, idx = _distill_inputs(rows, vocab, 12, 6)
    t, idx = torch.as_tensor(t).float().cuda(), torch.as_tensor(idx).cuda()
    for together in (False, True):
        b = Slices(torch, rows, {"s": vocab, "ds": vocab}, "bfloat16", gap, together)
        b.t["s"].copy_(torch.randn(rows, vocab, generator=torch.Generator("cuda").manual_seed(5), device="cuda"))
        loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
        v.vrcclDistillForward(b["s"], t, idx, loss, stats, rows, vocab, 12, "bfloat16", "float32", "int64", ldl=b.ld)
        v.vrcclDistillBackward(b["s"], t, idx, stats, loss, b["ds"], rows, vocab, 12, "bfloat16", "float32", "int64",
                               ldl=b.ld, ldd=b.ld)
        assert b.gaps_intact()
        got.append([t.clone() for t in (*b.t.values(), loss, stats)])
    assert all(torch.equal(a, c) for a, c in zip(*got))


# ------------------------------------------------------------ tensors through the binding

def test_views_are_taken_as_they_lie(torch, v):  # noqa: F811
    """Padded views without a row stride beside them give what the call with the stride gives."""
    rows, cols, outs, k = 30, 264, 72, 5
    g = torch.Generator("cuda").manual_seed(8)
    view = lambda n, pad=24: torch.randn(rows, n + pad, generator=g, device="cuda").bfloat16()[:, :n]  # noqa: E731
    x = view(cols)
    w = torch.randn(outs, cols + 8, generator=g, device="cuda").bfloat16()[:, :cols]
    out = []
    for strides in (True, False):
        kw = lambda **d: d if strides else {}  # noqa: E731
        y, z, r = (torch.zeros(rows, n + 16, device="cuda", dtype=torch.bfloat16)[:, :n] for n in (cols, outs, outs))
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        v.vrcclLayerNormForward(x, None, None, y, mean, rstd, rows, cols, "bfloat16", "float32", **kw(ldx=cols + 24, ldy=cols + 16))
        v.vrcclLinearForward(y, w, None, None, z, None, rows, outs, cols, torch.bfloat16, "silu",
                             **kw(ldx=cols + 16, ldw=cols + 8, ldy=outs + 16))
        t = (torch.arange(rows * 8, device="cuda").float() % 7).view(rows, 8)[:, :k]
        idx = (torch.arange(rows * 9, device="cuda") * 5 % outs).view(rows, 9)[:, :k]
        assert t.stride(0) == 8 and idx.stride(0) == 9
        loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
        v.vrcclDistillForward(z, t, idx, loss, stats, rows, outs, k, "bfloat16", "float32", "int64",
                              **kw(ldl=outs + 16, ldt=8, ldi=9))
        v.vrcclDistillBackward(z, t, idx, stats, loss, r, rows, outs, k, "bfloat16", "float32", "int64",
                               **kw(ldl=outs + 16, ldt=8, ldi=9, ldd=outs + 16))
        out.append([a.clone() for a in (y, mean, rstd, z, loss, stats, r)])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    with pytest.raises(ValueError):  # no row stride to be had
        v.vrcclLayerNormForward(x.t().contiguous().t(), None, None, x, None, None, rows, cols, "bfloat16", "float32")
    with pytest.raises(ValueError):  # a vector with gaps
        v.vrcclLayerNormForward(x, torch.ones(cols, 2, device="cuda")[:, 0], None, x, None, None, rows, cols, "bfloat16", "float32")
    # pinned memory on the host is the GPU's to write
    pinned = torch.zeros(rows, pin_memory=True)
    v.vrcclLayerNormForward(x, None, None, y, pinned, None, rows, cols, "bfloat16", "float32")
    torch.cuda.synchronize()
    assert torch.equal(pinned, mean.cpu())
