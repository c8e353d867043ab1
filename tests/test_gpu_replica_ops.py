"""The operators of a replica on the GPU, through the C ABI, against their
definitions in 64 bits (oracle/replica.py): values, gradients against the
formula and against differences, masks, strides, alignment, in place, other
streams and graphs.

Tolerances. U[t] is the largest relative error of one rounding to type t, and
EPS that of binary32. An output is within one rounding of its own type plus
what binary32 arithmetic loses on the way: the number of roundings a term goes
through, times EPS, times the sum of the absolute values that make up the
result (the quantity that bounds every intermediate sum). TINY covers results
below the type's normal range.
"""
import numpy as np
import pytest

from oracle import replica as o

pytestmark = pytest.mark.gpu

U = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 2.0 ** -120, "bfloat16": 2.0 ** -120, "float16": 2.0 ** -24}
EPS = 2.0 ** -24
FLOATS = ["float32", "bfloat16", "float16"]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def v():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_reduction_gb300 import build
    build.build()
    from ring_allreduce_reduction_gb300 import vrccl
    return vrccl


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


class Mat:
    """A [rows, cols] matrix inside a larger buffer: `offset` elements in front
    of it, `pad` after each row, all of them holding a canary value."""

    CANARY = 77.0

    def __init__(self, torch, rows, cols, dtype, values=None, pad=0, offset=0):
        self.rows, self.cols, self.ld, self.offset = rows, cols, cols + pad, offset
        self.buf = torch.full((offset + rows * self.ld + 8,), self.CANARY, device="cuda", dtype=getattr(torch, dtype))
        self.view = self.buf[offset:offset + rows * self.ld].view(rows, self.ld)[:, :cols]
        if values is not None:
            self.view.copy_(torch.as_tensor(values))
        self.ptr = self.buf.data_ptr() + offset * self.buf.element_size()

    def get(self):
        return self.view.double().cpu().numpy()

    def intact(self):
        a = self.buf.double().cpu().numpy()
        inside = np.zeros(a.size, bool)
        inside[self.offset:self.offset + self.rows * self.ld].reshape(self.rows, self.ld)[:, :self.cols] = True
        return bool((a[~inside] == self.CANARY).all())


def _rng(seed):
    return np.random.default_rng(seed)


def _close(got, want, tol, what):
    got, want = np.asarray(got), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: infinities"
    err = np.abs(got - want)[fine]
    tol = np.broadcast_to(tol, want.shape)[fine]
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err / np.maximum(tol, 1e-300)):.3g} tolerances"


# ------------------------------------------------------------ layer norm

def _norm_inputs(torch, rows, cols, dtype, ptype, pad, offset, seed, shift=0.25, affine=True):
    g = _rng(seed)
    x = Mat(torch, rows, cols, dtype, g.standard_normal((rows, cols)) * 1.5 + shift, pad, offset)
    dy = Mat(torch, rows, cols, dtype, g.standard_normal((rows, cols)), pad, offset)
    if not affine:
        return x, dy, None, None
    gamma = torch.as_tensor(1 + 0.2 * g.standard_normal(cols)).to("cuda", getattr(torch, ptype))
    beta = torch.as_tensor(0.2 * g.standard_normal(cols)).to("cuda", getattr(torch, ptype))
    return x, dy, gamma, beta


def _host(t):
    return t.double().cpu().numpy()


def _norm_check(torch, v, rows, cols, dtype, ptype, pad=0, offset=0, ypad=None, yoffset=None, affine=True, shift=0.25,
                eps=1e-5, seed=1):
    x, dy, gamma, beta = _norm_inputs(torch, rows, cols, dtype, ptype, pad, offset, seed, shift, affine)
    ypad, yoffset = pad if ypad is None else ypad, offset if yoffset is None else yoffset
    G = _host(gamma) if affine else np.ones(cols)
    B = _host(beta) if affine else np.zeros(cols)
    y = Mat(torch, rows, cols, dtype, None, ypad, yoffset)
    mean = torch.empty(rows, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    v.vrcclLayerNormForward(x.ptr, gamma, beta, y.ptr, mean, rstd, rows, cols, dtype, ptype, eps, ldx=x.ld, ldy=y.ld)
    X = x.get()
    wy, wm, wr = o.norm_forward(X, G, B, eps)
    # a sum of a row: at most 64 roundings a term (32 a thread, a warp's and a block's tree)
    steps = 64 * EPS
    amean = np.abs(X).mean(1)
    _close(_host(mean), wm, steps * amean, "mean")
    # an error of the mean adds its square to the variance; rstd takes half of the variance's relative error
    _close(_host(rstd), wr, wr * (steps + (steps * amean * wr) ** 2), "rstd")
    size = (np.abs(X - wm[:, None]) + amean[:, None]) * wr[:, None] * np.abs(G) + np.abs(B)
    _close(y.get(), wy, U[dtype] * np.abs(wy) * 1.01 + 2 * steps * size + TINY[dtype], "y")
    assert y.intact() and x.intact()

    # backward takes the statistics as they were saved
    M, R = _host(mean), _host(rstd)
    dx = Mat(torch, rows, cols, dtype, None, ypad, yoffset)
    dgamma = torch.empty(cols, device="cuda", dtype=getattr(torch, ptype))
    dbeta = torch.empty_like(dgamma)
    ws = torch.empty(max(16, v.vrcclLayerNormWorkspace(rows, cols)), device="cuda", dtype=torch.uint8)
    v.vrcclLayerNormBackward(dy.ptr, x.ptr, gamma, mean, rstd, dx.ptr, dgamma, dbeta, rows, cols, dtype, ptype, ws,
                             ws.numel(), lddy=dy.ld, ldx=x.ld, lddx=dx.ld)
    D = dy.get()
    wdx, wdg, wdb = o.norm_backward(D, X, G, M, R)
    xh = np.abs(X - M[:, None]) * R[:, None]
    xe = xh + np.abs(X) * R[:, None]  # what x - mean is made of
    g = np.abs(D * G)
    size = R[:, None] * (g + g.mean(1, keepdims=True) + xe * (g * xe).mean(1, keepdims=True))
    _close(dx.get(), wdx, U[dtype] * np.abs(wdx) * 1.01 + 2 * steps * size + TINY[dtype], "dx")
    # a column's sum: at most `rows` additions of a term
    down = (rows + 16) * EPS
    _close(_host(dgamma), wdg, U[ptype] * np.abs(wdg) * 1.01 + down * (np.abs(D) * xe).sum(0) + TINY[ptype], "dgamma")
    _close(_host(dbeta), wdb, U[ptype] * np.abs(wdb) * 1.01 + down * np.abs(D).sum(0) + TINY[ptype], "dbeta")
    assert dx.intact() and dy.intact()
    return x, dy, gamma, beta, M, R, dx


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (1, 8), (5, 33), (2, 256), (129, 264), (7, 512), (33, 768),
                                       (3, 1001), (5, 1024), (4, 1032), (311, 2048), (2, 4099), (2, 8192), (3, 8200),
                                       (2, 16384), (2, 16400), (1, 32768), (2, 32776), (3, 40001)])
def test_norm_sizes(torch, v, rows, cols, dtype):
    _norm_check(torch, v, rows, cols, dtype, dtype)


@pytest.mark.parametrize("pad,offset,ypad,yoffset", [(8, 0, 8, 0), (3, 0, 3, 0), (0, 1, 0, 1), (5, 3, 0, 0), (0, 0, 1, 8)])
@pytest.mark.parametrize("dtype,ptype", [("bfloat16", "float32"), ("float16", "bfloat16"), ("float32", "float16")])
@pytest.mark.parametrize("cols", [264, 1104])
def test_norm_strides_and_parameter_types(torch, v, dtype, ptype, cols, pad, offset, ypad, yoffset):
    _norm_check(torch, v, 37, cols, dtype, ptype, pad, offset, ypad, yoffset)


def test_norm_without_parameters(torch, v):
    _norm_check(torch, v, 19, 520, "bfloat16", "float32", affine=False)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad", [(400, 8200, 0), (333, 11440, 3), (310, 14336, 0), (170, 16384, 8), (457, 9001, 1)])
def test_norm_wide_rows_several_turns(torch, v, rows, cols, pad, dtype):
    """A block a row, more rows than multiprocessors, one shared-memory stage and several."""
    _norm_check(torch, v, rows, cols, dtype, "float32", pad)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad,ypad", [(1, 16, 0, 0), (3, 32, 8, 0), (1001, 64, 0, 8), (130, 128, 0, 0), (20003, 40, 0, 0),
                                               (9999, 200, 8, 16), (40001, 8, 0, 0)])
def test_norm_narrow_rows(torch, v, rows, cols, pad, ypad, dtype):
    """Several rows a warp, with lanes that hold nothing, and more rows than the grid takes at once."""
    _norm_check(torch, v, rows, cols, dtype, "float32", pad, 0, ypad, 0)


def test_norm_many_rows(torch, v):
    """More rows than blocks, several turns each."""
    _norm_check(torch, v, 5003, 264, "float16", "float32")
    _norm_check(torch, v, 2101, 1160, "bfloat16", "float32")


def test_norm_large_mean(torch, v):
    """A mean far from zero: squares are taken after it is subtracted."""
    _norm_check(torch, v, 16, 1024, "float32", "float32", shift=1000.0)


def test_norm_constant_rows(torch, v):
    """Zero variance: rstd is 1 / sqrt(eps), y is beta."""
    x = Mat(torch, 3, 96, "float32", np.full((3, 96), 0.5))
    y, beta = Mat(torch, 3, 96, "float32"), torch.arange(96, device="cuda", dtype=torch.float32)
    mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    v.vrcclLayerNormForward(x.ptr, None, beta, y.ptr, mean, rstd, 3, 96, "float32", "float32", 1e-4)
    assert np.array_equal(y.get(), np.tile(np.arange(96.0), (3, 1)))
    _close(_host(rstd), np.full(3, 100.0), 4 * EPS * 100, "rstd")


def test_norm_nan_stays_in_its_row(torch, v):
    a = _rng(3).standard_normal((6, 264))
    a[2, 5] = np.nan
    a[4, 7] = np.inf
    x, y = Mat(torch, 6, 264, "bfloat16", a), Mat(torch, 6, 264, "bfloat16")
    v.vrcclLayerNormForward(x.ptr, None, None, y.ptr, None, None, 6, 264, "bfloat16", "float32")
    assert np.array_equal(np.isnan(y.get()).all(1), [False, False, True, False, True, False])
    assert np.isfinite(y.get()[[0, 1, 3, 5]]).all()


@pytest.mark.parametrize("cols", [264, 1104, 33000])
def test_norm_in_place(torch, v, cols):
    rows = 40
    x, dy, gamma, beta = _norm_inputs(torch, rows, cols, "bfloat16", "float32", 0, 0, 5)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    apart = Mat(torch, rows, cols, "bfloat16")
    v.vrcclLayerNormForward(x.ptr, gamma, beta, apart.ptr, mean, rstd, rows, cols, "bfloat16", "float32")
    twin = Mat(torch, rows, cols, "bfloat16", x.get())
    v.vrcclLayerNormForward(twin.ptr, gamma, beta, twin.ptr, None, None, rows, cols, "bfloat16", "float32")
    assert np.array_equal(apart.get(), twin.get())
    ws = torch.empty(v.vrcclLayerNormWorkspace(rows, cols), device="cuda", dtype=torch.uint8)
    out = []
    for where in ("apart", "dy", "x"):
        cx, cd = Mat(torch, rows, cols, "bfloat16", x.get()), Mat(torch, rows, cols, "bfloat16", dy.get())
        dst = {"apart": Mat(torch, rows, cols, "bfloat16"), "dy": cd, "x": cx}[where]
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        v.vrcclLayerNormBackward(cd.ptr, cx.ptr, gamma, mean, rstd, dst.ptr, dg, db, rows, cols, "bfloat16", "float32",
                                 ws, ws.numel())
        out.append((dst.get(), _host(dg), _host(db)))
    for other in out[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(out[0], other))


def test_norm_no_rows(torch, v):
    dg = torch.full((16,), 5.0, device="cuda")
    db = torch.full((16,), 5.0, device="cuda")
    v.vrcclLayerNormForward(None, None, None, None, None, None, 0, 16, "float32", "float32")
    v.vrcclLayerNormBackward(None, None, None, None, None, None, dg, db, 0, 16, "float32", "float32")
    assert not dg.any() and not db.any()


def test_norm_one_gradient_only(torch, v):
    x, dy, gamma, beta, M, R, dx = _norm_check(torch, v, 50, 264, "float32", "float32")
    mean, rstd = torch.as_tensor(M).float().cuda(), torch.as_tensor(R).float().cuda()
    ws = torch.empty(v.vrcclLayerNormWorkspace(50, 264), device="cuda", dtype=torch.uint8)
    _, wdg, wdb = o.norm_backward(dy.get(), x.get(), _host(gamma), M, R)
    for which in (0, 1):
        out = torch.empty(264, device="cuda")
        again = Mat(torch, 50, 264, "float32")
        v.vrcclLayerNormBackward(dy.ptr, x.ptr, gamma, mean, rstd, again.ptr, None if which else out,
                                 out if which else None, 50, 264, "float32", "float32", ws, ws.numel())
        want = (wdg, wdb)[which]
        _close(_host(out), want, 2e-5 * (np.abs(want) + 50), "one gradient")
        assert np.array_equal(again.get(), dx.get())
    again = Mat(torch, 50, 264, "float32")
    v.vrcclLayerNormBackward(dy.ptr, x.ptr, gamma, mean, rstd, again.ptr, None, None, 50, 264, "float32", "float32")
    assert np.array_equal(again.get(), dx.get())


def test_norm_gradient_against_differences(torch, v):
    """The directional derivative of sum(dy * y) along random directions,
    by central differences of the definition in 64 bits."""
    rows, cols, eps, h = 9, 300, 1e-5, 1e-5
    x, dy, gamma, beta, M, R, dx = _norm_check(torch, v, rows, cols, "float32", "float32")
    X, D, G, B, g = x.get(), dy.get(), _host(gamma), _host(beta), _rng(9)
    for _ in range(4):
        d = g.standard_normal((rows, cols))
        f = lambda a: (D * o.norm_forward(a, G, B, eps)[0]).sum()  # noqa: E731
        slope = (f(X + h * d) - f(X - h * d)) / (2 * h)
        # the gradient's 128 roundings, and differences of second order with a third derivative of order one
        assert abs((dx.get() * d).sum() - slope) <= 1e-5 * (np.abs(dx.get() * d).sum() + 1)


# ------------------------------------------------------------ linear layer

def _linear_mats(torch, rows, outs, ins, dtype, pad, offset, seed):
    g = _rng(seed)
    x = Mat(torch, rows, ins, dtype, g.standard_normal((rows, ins)), pad, offset)
    w = Mat(torch, outs, ins, dtype, g.standard_normal((outs, ins)) / np.sqrt(max(1, ins)), pad, offset)
    bias = torch.as_tensor(0.5 * g.standard_normal(outs)).to("cuda", getattr(torch, dtype))
    r = Mat(torch, rows, outs, dtype, g.standard_normal((rows, outs)), pad, offset)
    dy = Mat(torch, rows, outs, dtype, g.standard_normal((rows, outs)), pad, offset)
    return x, w, bias, r, dy


def _scratch(torch, v, direction, rows, outs, ins, dtype, act):
    n = v.vrcclLinearWorkspace(direction, rows, outs, ins, dtype, act)
    return torch.empty(max(256, n), device="cuda", dtype=torch.uint8)


def _linear_check(torch, v, rows, outs, ins, dtype, act, pad=0, offset=0, bias=True, residual=True, save=True, seed=2):
    x, w, b, r, dy = _linear_mats(torch, rows, outs, ins, dtype, pad, offset, seed)
    b, r = b if bias else None, r if residual else None
    y = Mat(torch, rows, outs, dtype, None, pad, offset)
    z = Mat(torch, rows, outs, dtype, None, pad, offset) if save else None
    ws = _scratch(torch, v, "forward", rows, outs, ins, dtype, act)
    v.vrcclLinearForward(x.ptr, w.ptr, b, None if r is None else r.ptr, y.ptr, None if z is None else z.ptr, rows, outs,
                         ins, dtype, act, ws, ws.numel(), ldx=x.ld, ldw=w.ld, ldr=y.ld, ldy=y.ld, ldz=y.ld)
    X, W = x.get(), w.get()
    Bv, Rv = None if b is None else _host(b), None if r is None else r.get()
    wy, wz = o.linear_forward(X, W, Bv, Rv, act)
    u = U[dtype]
    # the sum's roundings, binary32 truncating in the tensor cores; activations have a slope below 1.2 and
    # are computed to a few units of their argument
    sums = (ins + 16) * 2 * EPS * (np.abs(X) @ np.abs(W).T + (0 if Bv is None else np.abs(Bv)))
    if z is not None:
        _close(z.get(), wz, u * np.abs(wz) * 1.01 + sums + TINY[dtype], "z")
        assert z.intact()
    own = 1.2 * sums + 16 * EPS * (1 + np.abs(wz)) + (0 if Rv is None else 2 * EPS * np.abs(Rv))
    _close(y.get(), wy, u * np.abs(wy) * 1.01 + own + TINY[dtype], "y")
    assert y.intact() and x.intact() and w.intact()
    assert v.vrcclReplicaGetAsyncError() == 0
    return x, w, z, dy


def _linear_back(torch, v, rows, outs, ins, dtype, act, pad=0, offset=0, seed=2):
    x, w, _, z, dy = _linear_mats(torch, rows, outs, ins, dtype, pad, offset, seed)  # any z will do
    dx, dw = Mat(torch, rows, ins, dtype, None, pad, offset), Mat(torch, outs, ins, dtype, None, pad, offset)
    db = torch.empty(outs, device="cuda", dtype=getattr(torch, dtype))
    ws = _scratch(torch, v, "backward", rows, outs, ins, dtype, act)
    v.vrcclLinearBackward(dy.ptr, z.ptr, x.ptr, w.ptr, dx.ptr, dw.ptr, db, rows, outs, ins, dtype, act, ws, ws.numel(),
                          lddy=dy.ld, ldz=z.ld, ldx=x.ld, ldw=w.ld, lddx=dx.ld, lddw=dw.ld)
    X, W, Z, D = x.get(), w.get(), z.get(), dy.get()
    wdx, wdw, wdb = o.linear_backward(D, Z, X, W, act)
    u = U[dtype]
    # |dz|, each off by one rounding to the type where an activation made it, and by a few units of its slope
    dz = np.abs(D) if act == "none" else np.abs(D * o.slope(Z, act))
    ez = 0 if act == "none" else u * 1.01 * dz + 32 * EPS * np.abs(D) * (1 + np.abs(Z)) + TINY[dtype]
    for got, want, err, size, n, what in (
            (dx.get(), wdx, ez @ np.abs(W) if act != "none" else 0, dz @ np.abs(W), outs, "dx"),
            (dw.get(), wdw, ez.T @ np.abs(X) if act != "none" else 0, dz.T @ np.abs(X), rows, "dw")):
        _close(got, want, u * np.abs(want) * 1.01 + err + (n + 16) * 2 * EPS * size + TINY[dtype], what)
    es = 0 if act == "none" else (32 * EPS * np.abs(D) * (1 + np.abs(Z))).sum(0)
    _close(_host(db), wdb, u * np.abs(wdb) * 1.01 + es + (rows + 16) * EPS * dz.sum(0) + TINY[dtype], "dbias")
    assert dx.intact() and dw.intact() and dy.intact() and z.intact()
    assert v.vrcclReplicaGetAsyncError() == 0
    return x, w, z, dy, dx, dw, db


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("rows,outs,ins", [(1, 1, 1), (1, 5, 64), (2, 64, 72), (3, 130, 513), (8, 96, 256), (9, 8, 8),
                                           (9, 1, 64), (17, 40, 24), (64, 64, 64), (128, 256, 64), (129, 257, 65),
                                           (200, 136, 1000), (333, 72, 328), (1000, 264, 136)])
def test_linear_sizes(torch, v, rows, outs, ins, dtype):
    _linear_check(torch, v, rows, outs, ins, dtype, "gelu")
    _linear_back(torch, v, rows, outs, ins, dtype, "gelu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 5, 160])
def test_linear_activations(torch, v, rows, act):
    _linear_check(torch, v, rows, 200, 128, "bfloat16", act)
    _linear_check(torch, v, rows, 200, 128, "float16", act, bias=False, residual=False, save=False)
    _linear_back(torch, v, rows, 200, 128, "float16", act)


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("rows", [1, 7, 70, 260])
def test_linear_strides(torch, v, rows, pad, offset):
    _linear_check(torch, v, rows, 88, 104, "bfloat16", "silu", pad, offset)
    _linear_back(torch, v, rows, 88, 104, "bfloat16", "silu", pad, offset)
    _linear_back(torch, v, rows, 88, 104, "float16", "none", pad, offset)


@pytest.mark.parametrize("rows,outs,ins,pad", [(129, 257, 65, 7), (300, 1001, 33, 23), (65, 63, 127, 1)])
def test_linear_ragged_rows_on_vector_boundaries(torch, v, rows, outs, ins, pad):
    """Rows that end inside a vector but start on one: nothing past a row's end is written."""
    for act in ("none", "relu"):
        _linear_check(torch, v, rows, outs, ins, "bfloat16", act, pad)
        _linear_back(torch, v, rows, outs, ins, "bfloat16", act, pad)


@pytest.mark.parametrize("rows,outs,ins", [(2048, 2560, 192), (4100, 1300, 320), (300, 5000, 64), (24, 6000, 2048),
                                           (100, 100, 8192)])
def test_linear_many_tiles(torch, v, rows, outs, ins):
    """Several tiles a block, every tile width, a long contraction."""
    _linear_check(torch, v, rows, outs, ins, "bfloat16", "none", residual=False, save=False)
    _linear_back(torch, v, rows, outs, ins, "bfloat16", "none")


@pytest.mark.parametrize("rows,outs,ins", [(744, 3584, 600), (750, 3561, 611)])
def test_linear_tiles_of_192_columns(torch, v, rows, outs, ins):
    for act in ("gelu_tanh", "none"):
        _linear_check(torch, v, rows, outs, ins, "bfloat16", act)
    _linear_check(torch, v, rows, outs, ins, "float16", "silu", 5, 1)


@pytest.mark.parametrize("rows,outs,ins", [(3, 4096, 512), (5, 1000, 1000), (16, 1024, 4096), (20, 130, 2056), (32, 136, 136),
                                           (33, 1000, 2048), (64, 64, 4096), (65, 520, 1536), (128, 1024, 2048),
                                           (250, 300, 1100), (512, 512, 4096), (130, 72, 4104)])
def test_linear_split_contractions(torch, v, rows, outs, ins):
    """Few rows or few tiles against a long contraction: every way a call is cut."""
    for act in ("silu", "none"):
        _linear_check(torch, v, rows, outs, ins, "bfloat16", act)
    _linear_check(torch, v, rows, outs, ins, "float16", "gelu", 8, 8)
    _linear_back(torch, v, rows, outs, ins, "bfloat16", "none")


def test_linear_residual_in_place(torch, v):
    for rows in (3, 150):
        x, w, b, r, _ = _linear_mats(torch, rows, 136, 64, "bfloat16", 0, 0, 4)
        y = Mat(torch, rows, 136, "bfloat16")
        v.vrcclLinearForward(x.ptr, w.ptr, b, r.ptr, y.ptr, None, rows, 136, 64, "bfloat16", "relu")
        v.vrcclLinearForward(x.ptr, w.ptr, b, r.ptr, r.ptr, None, rows, 136, 64, "bfloat16", "relu")
        assert np.array_equal(y.get(), r.get())


@pytest.mark.parametrize("rows", [4, 140])
def test_linear_nan_and_infinity_stay_in_their_rows(torch, v, rows):
    """Rows beyond the matrix's end are not read, and a row's NaN reaches that row alone."""
    x, w, b, _, _ = _linear_mats(torch, rows, 72, 40, "bfloat16", 0, 0, 6)
    x.view[1, 3] = float("nan")
    x.view[rows - 1, 0] = float("inf")
    y = Mat(torch, rows, 72, "bfloat16")
    v.vrcclLinearForward(x.ptr, w.ptr, b, None, y.ptr, None, rows, 72, 40, "bfloat16", "none")
    got = y.get()
    assert np.isnan(got[1]).all() and not np.isfinite(got[rows - 1]).any()
    keep = [i for i in range(rows) if i not in (1, rows - 1)]
    assert np.isfinite(got[keep]).all()


def test_linear_fp16_overflow_is_infinite(torch, v):
    x, w = Mat(torch, 130, 64, "float16", np.full((130, 64), 250.0)), Mat(torch, 64, 64, "float16", np.full((64, 64), 250.0))
    y = Mat(torch, 130, 64, "float16")
    v.vrcclLinearForward(x.ptr, w.ptr, None, None, y.ptr, None, 130, 64, 64, "float16", "none")
    assert np.isposinf(y.get()).all()


@pytest.mark.parametrize("rows,outs,ins", [(0, 8, 8), (8, 0, 8), (20, 8, 0), (0, 8, 0)])
def test_linear_empty(torch, v, rows, outs, ins):
    x, w, b, r, dy = _linear_mats(torch, rows, outs, ins, "bfloat16", 0, 0, 7)
    y = Mat(torch, rows, outs, "bfloat16")
    v.vrcclLinearForward(x.ptr, w.ptr, b, r.ptr, y.ptr, None, rows, outs, ins, "bfloat16", "relu")
    wy, _ = o.linear_forward(x.get(), w.get(), _host(b), r.get(), "relu")
    _close(y.get(), wy, U["bfloat16"] * np.abs(wy) * 1.01 + 4 * EPS, "y")
    dx, dw = Mat(torch, rows, ins, "bfloat16"), Mat(torch, outs, ins, "bfloat16")
    db = torch.full((outs,), 3.0, device="cuda", dtype=torch.bfloat16)
    ws = _scratch(torch, v, "backward", rows, outs, ins, "bfloat16", "relu")
    v.vrcclLinearBackward(dy.ptr, r.ptr, x.ptr, w.ptr, dx.ptr, dw.ptr, db, rows, outs, ins, "bfloat16", "relu", ws,
                          ws.numel())
    assert not dx.get().any() and not dw.get().any()
    if rows == 0:
        assert not db.any()


def test_linear_single_gradients(torch, v):
    rows, outs, ins = 150, 72, 136
    x, w, z, dy, dx, dw, db = _linear_back(torch, v, rows, outs, ins, "bfloat16", "gelu_tanh")
    ws = _scratch(torch, v, "backward", rows, outs, ins, "bfloat16", "gelu_tanh")
    for which in range(3):
        a, c = Mat(torch, rows, ins, "bfloat16"), Mat(torch, outs, ins, "bfloat16")
        e = torch.empty_like(db)
        v.vrcclLinearBackward(dy.ptr, z.ptr, x.ptr if which == 1 else None, w.ptr if which == 0 else None,
                              a.ptr if which == 0 else None, c.ptr if which == 1 else None, e if which == 2 else None,
                              rows, outs, ins, "bfloat16", "gelu_tanh", ws, ws.numel())
        got, want = ((a.get(), dx.get()), (c.get(), dw.get()), (_host(e), _host(db)))[which]
        assert np.array_equal(got, want)


@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
def test_linear_gradient_against_differences(torch, v, act):
    """Directional derivatives of sum(dy * y) in x, w and bias, by central differences in 64 bits."""
    rows, outs, ins, h = 40, 48, 56, 1e-5
    x, w, z, dy = _linear_check(torch, v, rows, outs, ins, "float16", act, bias=False, residual=False)
    dx, dw = Mat(torch, rows, ins, "float16"), Mat(torch, outs, ins, "float16")
    db = torch.empty(outs, device="cuda", dtype=torch.float16)
    ws = _scratch(torch, v, "backward", rows, outs, ins, "float16", act)
    v.vrcclLinearBackward(dy.ptr, z.ptr, x.ptr, w.ptr, dx.ptr, dw.ptr, db, rows, outs, ins, "float16", act, ws, ws.numel())
    X, W, D, g = x.get(), w.get(), dy.get(), _rng(11)
    f = lambda a, b, c: (D * o.linear_forward(a, b, c, None, act)[0]).sum()  # noqa: E731
    zero = np.zeros(outs)
    for grad, at in ((dx.get(), 0), (dw.get(), 1), (_host(db), 2)):
        d = g.standard_normal(grad.shape)
        step = [h * d if i == at else 0 for i in range(3)]
        slope = (f(X + step[0], W + step[1], zero + step[2]) - f(X - step[0], W - step[1], zero - step[2])) / (2 * h)
        # z and dz are each rounded to the type (slopes change by less than their argument), and the gradient once
        # more; every element's error is independent of d's sign: bounded by the sum of absolutes
        size = np.abs(D).max() * (np.abs(X) @ np.abs(W).T + 1).max()
        assert abs((grad * d).sum() - slope) <= U["float16"] * 4 * (np.abs(grad * d).sum() + size * np.abs(d).max() * 8)


# ------------------------------------------------------------ distillation

def _distill_inputs(rows, vocab, k, seed, scale=2.5):
    g = _rng(seed)
    s = g.standard_normal((rows, vocab)) * scale
    t = np.sort(g.standard_normal((rows, k)) * 3 + 8, 1)[:, ::-1].copy()
    idx = np.stack([g.permutation(vocab)[:k] if k <= vocab else g.integers(0, vocab, k) for _ in range(rows)])
    return s, t, idx.astype(np.int64)


def _distill_check(torch, v, s, t, idx, dtype, ttype="float32", itype="int64", T=1.0, pad=0, offset=0, dpad=None,
                   doffset=None, inplace=False, broadcast=False):
    rows, vocab = s.shape
    k = t.shape[1]
    S = Mat(torch, rows, vocab, dtype, s, pad, offset)
    Te = Mat(torch, rows, k, ttype, t, 1, 1)
    I = torch.as_tensor(idx).to("cuda", getattr(torch, itype)).contiguous()
    loss = torch.full((rows,), 9.0, device="cuda")
    stats = torch.full((rows, 2), 9.0, device="cuda")
    v.vrcclDistillForward(S.ptr, Te.ptr, I, loss, stats, rows, vocab, k, dtype, ttype, itype, T, ldl=S.ld, ldt=Te.ld)
    s, t = S.get(), Te.get()
    with np.errstate(invalid="ignore", divide="ignore"):
        wl, ws = o.distill_forward(s, t, idx, T)
    # logs of sums of exponentials: an exponential's relative error is its argument's absolute one (its size times a
    # few EPS) plus the exponential's own 2^-21; the loss adds log p and log q weighted by p
    finite = np.where(np.isfinite(s), s, 0.0)
    span = np.minimum((finite.max(1) - finite.min(1)) / T, 200.0)
    e = 2.0 ** -20 + 16 * EPS * (span + np.log(vocab + 1))
    tf = np.where(np.isfinite(t), t, 0.0)
    tspan = (tf.max(1) - tf.min(1)) / T if k else 0 * span
    far = np.zeros(rows)
    for r in range(rows):
        kept = (idx[r] >= 0) & (idx[r] < vocab)
        far[r] = max([0.0] + [abs(x - finite[r].max()) / T for x in finite[r][idx[r][kept]]])
    el = T * T * (2 * e + 32 * EPS * (tspan + np.minimum(far, 1e30)))
    _close(_host(stats)[:, 0], ws[:, 0], 0, "largest logit")
    _close(_host(stats)[:, 1], ws[:, 1], e + EPS * np.abs(ws[:, 1]), "log of the sum")
    _close(_host(loss), wl, el + 16 * EPS * np.abs(np.where(np.isfinite(wl), wl, 0)), "loss")

    g = _rng(77).standard_normal(1 if broadcast else rows)
    dl = torch.as_tensor(g).float().cuda()
    ref = np.broadcast_to(_host(dl), (rows,))
    D = S if inplace else Mat(torch, rows, vocab, dtype, None, pad if dpad is None else dpad,
                              offset if doffset is None else doffset)
    v.vrcclDistillBackward(S.ptr, Te.ptr, I, stats, dl, D.ptr, rows, vocab, k, dtype, ttype, itype, T,
                           dloss_stride=0 if broadcast else 1, ldl=S.ld, ldt=Te.ld, ldd=D.ld)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        wd = o.distill_backward(s, t, idx, ref, T)
        q = np.exp((s - ws[:, :1]) / T - ws[:, 1:])
    q = np.where(np.isfinite(q), q, 0)
    p = q * 0
    for r in range(rows):
        kept = (idx[r] >= 0) & (idx[r] < vocab) & ~(t[r] == -np.inf)
        if kept.any():
            x = np.exp((t[r][kept] - t[r][kept].max()) / T)
            np.add.at(p[r], idx[r][kept], x / x.sum())
    # q and p each carry their exponent's error
    tol = np.abs(ref)[:, None] * T * (q * (3 * e)[:, None] + p * (2.0 ** -20 + 64 * EPS * (1 + tspan))[:, None])
    _close(D.get(), wd, U[dtype] * np.abs(wd) * 1.01 + tol + TINY[dtype] * 2, "dlogits")
    assert D.intact() and S.intact()
    return _host(loss), D.get()


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (2, 7, 3), (3, 64, 64), (1, 4096, 8), (5, 4099, 100), (40, 1000, 1),
                                          (2, 50001, 33), (3, 32768, 1024), (1, 131072, 64), (700, 520, 16)])
def test_distill_sizes(torch, v, rows, vocab, k, dtype):
    _distill_check(torch, v, *_distill_inputs(rows, vocab, k, 1), dtype)


@pytest.mark.parametrize("ttype", FLOATS)
@pytest.mark.parametrize("itype", ["int32", "int64"])
@pytest.mark.parametrize("T", [0.5, 1.0, 4.0])
def test_distill_types_and_temperatures(torch, v, ttype, itype, T):
    _distill_check(torch, v, *_distill_inputs(6, 2003, 20, 2), "bfloat16", ttype, itype, T)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("pad,offset,dpad,doffset", [(8, 0, 8, 0), (3, 0, 3, 0), (0, 1, 0, 1), (5, 3, 0, 0), (0, 0, 1, 8)])
def test_distill_strides(torch, v, dtype, pad, offset, dpad, doffset):
    for rows, vocab in ((9, 1003), (2, 70000)):
        _distill_check(torch, v, *_distill_inputs(rows, vocab, 17, 3), dtype, T=2.0, pad=pad, offset=offset, dpad=dpad,
                       doffset=doffset)


@pytest.mark.parametrize("rows,vocab", [(9, 1003), (2, 131072), (300, 5000)])
def test_distill_in_place_and_broadcast_gradient(torch, v, rows, vocab):
    args = _distill_inputs(rows, vocab, 40, 4)
    _, apart = _distill_check(torch, v, *args, "bfloat16", T=2.0, broadcast=True)
    _, here = _distill_check(torch, v, *args, "bfloat16", T=2.0, broadcast=True, inplace=True)
    assert np.array_equal(apart, here)


def test_distill_missing_entries_and_empty_rows(torch, v):
    """Indices outside the vocabulary and teacher logits of -inf are passed
    over; a row with none left has loss and gradient zero, whatever it holds."""
    s, t, idx = _distill_inputs(8, 3001, 12, 5)
    idx[0] = -1
    idx[1, ::2] = -1
    idx[2, 3:] = 3001
    t[3, 5:] = -np.inf
    t[4] = -np.inf
    idx[5, 0] = 1 << 40
    s[0] = np.nan
    s[4, 7] = np.inf
    loss, d = _distill_check(torch, v, s, t, idx, "float32")
    assert loss[0] == 0 and loss[4] == 0 and not d[[0, 4]].any()


def test_distill_shared_indices_add_up(torch, v):
    s, t, idx = _distill_inputs(4, 999, 30, 6)
    idx[0, :] = 5
    idx[1, 10:20] = idx[1, 0]
    _distill_check(torch, v, s, t, idx, "float32")


@pytest.mark.parametrize("dtype", FLOATS)
def test_distill_masked_logits(torch, v, dtype):
    """A vocabulary masked with -inf or the type's lowest value, also on both sides of the temperature."""
    lowest = float(torch.finfo(getattr(torch, dtype)).min)
    for T in (0.5, 2.0):
        s, t, idx = _distill_inputs(5, 2048, 6, 7)
        s[0, 100:] = -np.inf
        idx[0] = np.arange(6)
        s[1, 100:] = lowest
        idx[1] = np.arange(6)
        s[2, :] = lowest       # every entry equal: uniform
        s[3, 1:] = -np.inf     # one entry left
        idx[3] = 0
        _distill_check(torch, v, s, t, idx, dtype, T=T)


def test_distill_teacher_where_the_student_has_none(torch, v):
    """log q = -inf at an entry with p > 0: the loss is infinite, the gradient is not."""
    s, t, idx = _distill_inputs(2, 500, 4, 8)
    s[0, idx[0, 1]] = -np.inf
    loss, d = _distill_check(torch, v, s, t, idx, "float32")
    assert np.isposinf(loss[0]) and np.isfinite(loss[1]) and np.isfinite(d).all()


def test_distill_nan_stays_in_its_row(torch, v):
    s, t, idx = _distill_inputs(5, 700, 4, 9)
    s[1, 30] = np.nan
    t[3, 2] = np.nan
    S = Mat(torch, 5, 700, "float32", s)
    loss, stats = torch.empty(5, device="cuda"), torch.empty(5, 2, device="cuda")
    v.vrcclDistillForward(S.ptr, torch.as_tensor(t).float().cuda(), torch.as_tensor(idx).cuda(), loss, stats, 5, 700, 4,
                          "float32", "float32", "int64")
    assert np.array_equal(np.isnan(_host(loss)), [False, True, False, True, False])


def test_distill_large_logits(torch, v):
    """Statistics kept as maximum and logarithm lose nothing to a large common part."""
    s, t, idx = _distill_inputs(3, 1000, 8, 10)
    _distill_check(torch, v, s + 4096.0, t + 4096.0, idx, "float32")


def test_distill_gradient_against_differences(torch, v):
    rows, vocab, k, T, h = 3, 400, 9, 2.0, 1e-5
    s, t, idx = _distill_inputs(rows, vocab, k, 11)
    S = Mat(torch, rows, vocab, "float32", s)
    s = S.get()
    t32 = torch.as_tensor(t).float().cuda()
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    I, one = torch.as_tensor(idx).cuda(), torch.ones(1, device="cuda")
    v.vrcclDistillForward(S.ptr, t32, I, loss, stats, rows, vocab, k, "float32", "float32", "int64", T)
    D = Mat(torch, rows, vocab, "float32")
    v.vrcclDistillBackward(S.ptr, t32, I, stats, one, D.ptr, rows, vocab, k, "float32", "float32", "int64", T, dloss_stride=0)
    g = _rng(12)
    for _ in range(4):
        d = g.standard_normal((rows, vocab))
        f = lambda a: o.distill_forward(a, _host(t32), idx, T)[0].sum()  # noqa: E731
        slope = (f(s + h * d) - f(s - h * d)) / (2 * h)
        assert abs((D.get() * d).sum() - slope) <= 2e-5 * np.abs(D.get() * d).sum() + 1e-7


def test_distill_no_entries(torch, v):
    """k = 0, and rows = 0."""
    S = Mat(torch, 3, 50, "bfloat16", np.ones((3, 50)))
    loss, stats = torch.ones(3, device="cuda"), torch.ones(3, 2, device="cuda")
    v.vrcclDistillForward(S.ptr, None, None, loss, stats, 3, 50, 0, "bfloat16", "float32", "int32")
    D = Mat(torch, 3, 50, "bfloat16", np.ones((3, 50)), pad=6)
    v.vrcclDistillBackward(S.ptr, None, None, stats, loss, D.ptr, 3, 50, 0, "bfloat16", "float32", "int32", ldd=56)
    assert not loss.any() and not stats.any() and not D.get().any() and D.intact()
    v.vrcclDistillForward(None, None, None, None, None, 0, 50, 4, "bfloat16", "float32", "int32")


# ------------------------------------------------------------ far apart

@pytest.mark.parametrize("gap", [0, 3])
def test_offsets_beyond_32_bits(torch, v, gap):
    """Rows so far apart that the last one's offset exceeds 2^32 elements."""
    rows, ld = 2100, (1 << 21) + gap
    buf = torch.empty(rows * ld, device="cuda", dtype=torch.bfloat16)
    far = lambda cols: buf.view(rows, ld)[:, :cols]  # noqa: E731
    g, u = _rng(41), U["bfloat16"]
    a = torch.as_tensor(g.standard_normal((rows, 264))).cuda().bfloat16()
    x = far(264).copy_(a)
    # layer norm, in place, forward and backward, against the same rows side by side
    near, back = torch.empty_like(a), torch.empty_like(a)
    mean, rstd, dg, db, dg2, db2 = (torch.empty(n, device="cuda") for n in (rows, rows, 264, 264, 264, 264))
    v.vrcclLayerNormForward(a, None, None, near, mean, rstd, rows, 264, "bfloat16", "float32")
    ws = torch.empty(v.vrcclLayerNormWorkspace(rows, 264), device="cuda", dtype=torch.uint8)
    v.vrcclLayerNormBackward(a, a, None, mean, rstd, back, dg, db, rows, 264, "bfloat16", "float32", ws, ws.numel())
    v.vrcclLayerNormBackward(x, a, None, mean, rstd, x, dg2, db2, rows, 264, "bfloat16", "float32", ws, ws.numel(),
                             lddy=ld, lddx=ld)
    _close(_host(x), _host(back), 2 * u * np.abs(_host(back)) + 64 * EPS, "dx")
    _close(_host(dg2), _host(dg), rows * EPS * np.abs(_host(a) ** 2).sum(0), "dgamma")
    x.copy_(a)
    v.vrcclLayerNormForward(x, None, None, x, None, None, rows, 264, "bfloat16", "float32", ldx=ld, ldy=ld)
    _close(_host(x), _host(near), 2 * u * np.abs(_host(near)) + 64 * EPS, "y")
    # linear layer
    w = torch.as_tensor(g.standard_normal((72, 264)) / 16).cuda().bfloat16()
    x.copy_(a)
    y, y2 = torch.empty(rows, 72, device="cuda", dtype=torch.bfloat16), torch.empty(rows, 72, device="cuda", dtype=torch.bfloat16)
    ws = _scratch(torch, v, "backward", rows, 72, 264, "bfloat16", "none")
    v.vrcclLinearForward(a, w, None, None, y, None, rows, 72, 264, "bfloat16")
    v.vrcclLinearForward(x, w, None, None, y2, None, rows, 72, 264, "bfloat16", "none", ws, ws.numel(), ldx=ld)
    assert torch.equal(y, y2)
    dw, dw2 = torch.empty_like(w), torch.empty_like(w)
    v.vrcclLinearBackward(y, None, a, None, None, dw, None, rows, 72, 264, "bfloat16", "none", ws, ws.numel())
    v.vrcclLinearBackward(y, None, x, None, None, dw2, None, rows, 72, 264, "bfloat16", "none", ws, ws.numel(), ldx=ld)
    assert torch.equal(dw, dw2)
    v.vrcclLinearBackward(y, None, None, w, back, None, None, rows, 72, 264, "bfloat16", "none", ws, ws.numel())
    v.vrcclLinearBackward(y, None, None, w, x, None, None, rows, 72, 264, "bfloat16", "none", ws, ws.numel(), lddx=ld)
    assert torch.equal(back, x)
    # distillation
    x.copy_(a)
    t = torch.as_tensor(g.standard_normal((rows, 5))).float().cuda()
    idx = torch.as_tensor(g.integers(0, 264, (rows, 5))).cuda()
    one = torch.ones(1, device="cuda")
    out = []
    for s, stride in ((a.clone(), 264), (x, ld)):
        loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
        v.vrcclDistillForward(s, t, idx, loss, stats, rows, 264, 5, "bfloat16", "float32", "int64", ldl=stride)
        v.vrcclDistillBackward(s, t, idx, stats, one, s, rows, 264, 5, "bfloat16", "float32", "int64", dloss_stride=0,
                               ldl=stride, ldd=stride)
        out.append((_host(loss), _host(s)))
    _close(out[1][0], out[0][0], 1e-5 * np.abs(out[0][0]) + 1e-6, "loss")
    _close(out[1][1], out[0][1], 2 * u * np.abs(out[0][1]) + 1e-6, "dlogits")


# ------------------------------------------------------------ streams, graphs, repeats

def _everything(torch, v, stream=None):
    """One pass of each operator on fixed inputs; the outputs."""
    rows, cols, outs, vocab, k = 150, 264, 136, 1000, 10
    x, dy, gamma, beta = _norm_inputs(torch, rows, cols, "bfloat16", "float32", 0, 0, 31)
    X, w, b, r, g = _linear_mats(torch, rows, outs, cols, "bfloat16", 0, 0, 32)
    s, t, idx = _distill_inputs(rows, vocab, k, 33)
    S, t, idx = Mat(torch, rows, vocab, "bfloat16", s), torch.as_tensor(t).float().cuda(), torch.as_tensor(idx).cuda()
    y, dx, ly, lz = (Mat(torch, rows, n, "bfloat16") for n in (cols, cols, outs, outs))
    ldx, ldw, ds = Mat(torch, rows, cols, "bfloat16"), Mat(torch, outs, cols, "bfloat16"), Mat(torch, rows, vocab, "bfloat16")
    f = {n: torch.empty(sz, device="cuda") for n, sz in (("mean", rows), ("rstd", rows), ("dg", cols), ("db", cols),
                                                         ("loss", rows), ("stats", (rows, 2)))}
    db = torch.empty(outs, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(max(v.vrcclLayerNormWorkspace(rows, cols), v.vrcclLinearWorkspace("backward", rows, outs, cols, "bfloat16", "gelu")),
                     device="cuda", dtype=torch.uint8)
    torch.cuda.synchronize()

    def go():
        kw = {"stream": stream}
        v.vrcclLayerNormForward(x.ptr, gamma, beta, y.ptr, f["mean"], f["rstd"], rows, cols, "bfloat16", "float32", **kw)
        v.vrcclLinearForward(y.ptr, w.ptr, b, r.ptr, ly.ptr, lz.ptr, rows, outs, cols, "bfloat16", "gelu", **kw)
        v.vrcclLinearBackward(g.ptr, lz.ptr, y.ptr, w.ptr, ldx.ptr, ldw.ptr, db, rows, outs, cols, "bfloat16", "gelu", ws,
                              ws.numel(), **kw)
        v.vrcclLayerNormBackward(ldx.ptr, x.ptr, gamma, f["mean"], f["rstd"], dx.ptr, f["dg"], f["db"], rows, cols,
                                 "bfloat16", "float32", ws, ws.numel(), **kw)
        v.vrcclDistillForward(S.ptr, t, idx, f["loss"], f["stats"], rows, vocab, k, "bfloat16", "float32", "int64", 2.0, **kw)
        v.vrcclDistillBackward(S.ptr, t, idx, f["stats"], f["loss"], ds.ptr, rows, vocab, k, "bfloat16", "float32",
                               "int64", 2.0, **kw)

    def out():
        torch.cuda.synchronize()
        return [m.get() for m in (y, ly, lz, ldx, ldw, dx, ds)] + [_host(a) for a in (*f.values(), db)]

    return go, out


def test_same_bits_again_on_another_stream_and_in_a_graph(torch, v):
    go, out = _everything(torch, v)
    go()
    first = out()
    go()
    assert all(np.array_equal(a, b) for a, b in zip(first, out()))
    side = torch.cuda.Stream()
    go, out = _everything(torch, v, side)
    go()
    assert all(np.array_equal(a, b) for a, b in zip(first, out()))
    graph = torch.cuda.CUDAGraph()
    go, out = _everything(torch, v)
    with torch.cuda.graph(graph):
        go()
    graph.replay()
    assert all(np.array_equal(a, b) for a, b in zip(first, out()))
