"""The replica's RMS norm on the GPU against its definition in 64 bits
(oracle/replica.py): sums, values, 8-bit codes and scales, gradients against
the formula and against differences, strides, alignment, in place, graphs.
Helpers and U, EPS, TINY as in test_gpu_replica_ops.py."""
import numpy as np
import pytest

from oracle import replica as o
from test_gpu_replica_ops import EPS, FLOATS, TINY, U, Mat, _close, _host, _rng, torch, v  # noqa: F401

pytestmark = pytest.mark.gpu

STEPS = 64 * EPS  # a row's sum: at most 64 roundings a term (16 a thread, a warp's and a block's tree), the root's among them
LARGEST = {"int8": 127.0, "e4m3": 448.0}


def _gamma(torch, g, cols, ptype):  # noqa: F811
    return torch.as_tensor(1 + 0.2 * g.standard_normal(cols)).to("cuda", getattr(torch, ptype))


def _codes(torch, rows, cols, quant, pad):  # noqa: F811
    td = torch.int8 if quant == "int8" else torch.float8_e4m3fn
    buf = torch.full((rows, cols + pad), 77, device="cuda", dtype=torch.uint8)
    return buf, buf.view(td)[:, :cols]


def _check_codes(codes, scales, y, quant, group, extra):
    """`extra`: the relative error of y that the norm itself may have."""
    want = o.group_scales(y, quant, group)
    _close(scales, want, (extra + 4 * EPS) * want, "scales")
    wide = np.repeat(scales, group or y.shape[1], 1)[:, :y.shape[1]]
    at = y / wide
    step = np.ones_like(at) if quant == "int8" else 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.maximum(np.abs(at), np.abs(codes)), 1e-30))) - 3, -9)
    # half a step, and what the value was off before it was rounded
    off = np.abs(codes - at) - step / 2 - (extra + 4 * EPS) * np.abs(at)
    assert off.max() <= 0, f"codes: off by {off.max():.3g} beyond half a step"
    assert np.abs(codes).max() <= LARGEST[quant]


def _forward(torch, v, rows, cols, dtype, ptype="float32", pad=0, offset=0, residual=True, affine=True, quant=None, group=0,  # noqa: F811
             with_y=True, eps=1e-5, scale=1.0, opad=None, oskew=None, seed=1):
    g = _rng(seed)
    x = Mat(torch, rows, cols, dtype, scale * g.standard_normal((rows, cols)), pad, offset)
    r = Mat(torch, rows, cols, dtype, scale * g.standard_normal((rows, cols)), pad, offset) if residual else None
    gamma = _gamma(torch, g, cols, ptype) if affine else None
    opad, oskew = pad if opad is None else opad, offset if oskew is None else oskew
    s = Mat(torch, rows, cols, dtype, None, opad, oskew)
    y = Mat(torch, rows, cols, dtype, None, opad, oskew) if with_y else None
    rstd = torch.empty(rows, device="cuda")
    more = {}
    if quant:
        buf, codes = _codes(torch, rows, cols, quant, pad)
        groups = -(-cols // group) if group else 1
        scales = torch.empty(rows, groups + 1, device="cuda")[:, :groups]
        more = dict(codes=codes, scales=scales, quant=quant, group=group)
    v.vrcclRmsNormForward(x.ptr, r.ptr if residual else None, gamma, s.ptr, y.ptr if y else None, rstd, rows, cols, dtype, ptype,
                          eps, ldx=x.ld, ldr=r.ld if residual else None, lds=s.ld, ldy=y.ld if y else None, **more)
    sums = x.view.float() + r.view.float() if residual else x.view
    assert torch.equal(s.view, sums.to(getattr(torch, dtype)))
    wy, wr = o.rms_forward(s.get(), _host(gamma) if affine else np.ones(cols), eps)
    _close(_host(rstd), wr, STEPS * wr, "rstd")
    if y:
        _close(y.get(), wy, (U[dtype] * 1.01 + 2 * STEPS) * np.abs(wy) + TINY[dtype], "y")
        assert y.intact()
    if quant:
        _check_codes(_host(codes.float()), _host(scales), wy, quant, group, 2 * STEPS)
        assert (buf[:, cols:] == 77).all()
    assert s.intact() and x.intact()


def _backward(torch, v, rows, cols, dtype, ptype="float32", pad=0, offset=0, dsum=True, affine=True, dgamma=True, opad=None,  # noqa: F811
              oskew=None, seed=2):
    g = _rng(seed)
    s, dy = (Mat(torch, rows, cols, dtype, g.standard_normal((rows, cols)), pad, offset) for _ in range(2))
    ds = Mat(torch, rows, cols, dtype, g.standard_normal((rows, cols)), pad, offset) if dsum else None
    gamma = _gamma(torch, g, cols, ptype) if affine else None
    dx = Mat(torch, rows, cols, dtype, None, pad if opad is None else opad, offset if oskew is None else oskew)
    dg = torch.empty(cols, device="cuda", dtype=getattr(torch, ptype)) if dgamma else None
    G = _host(gamma) if affine else np.ones(cols)
    S, D, add = s.get(), dy.get(), ds.get() if dsum else np.zeros((rows, cols))
    rstd = torch.as_tensor(o.rms_forward(S, G, 1e-5)[1]).float().cuda()
    ws = torch.empty(v.vrcclRmsNormWorkspace(rows, cols) + 16, device="cuda", dtype=torch.uint8).fill_(255)
    v.vrcclRmsNormBackward(dy.ptr, ds.ptr if dsum else None, s.ptr, gamma, rstd, dx.ptr, dg, rows, cols, dtype, ptype,
                           ws if dgamma else None, ws.numel() - 16 if dgamma else 0, lddy=dy.ld, lddsum=ds.ld if dsum else None,
                           lds=s.ld, lddx=dx.ld)
    assert (ws[-16:] == 255).all()
    R = _host(rstd)[:, None]
    wx, wg = o.rms_backward(D, add, S, G, _host(rstd))
    xh, gd = np.abs(S * R), np.abs(D * G)
    size = np.abs(add) + R * (gd + xh * (gd * xh).mean(1, keepdims=True))
    _close(dx.get(), wx, U[dtype] * 1.01 * np.abs(wx) + 2 * STEPS * size + TINY[dtype], "dx")
    assert dx.intact()
    if dgamma:
        # products of two roundings each, added one after another at worst
        _close(_host(dg), wg, U[ptype] * 1.01 * np.abs(wg) + (rows + 16) * EPS * np.abs(D * S * R).sum(0) + TINY[ptype], "dgamma")


SHAPES = [(1, 1, 0, 0), (1, 8, 0, 0), (3, 7, 0, 1), (40, 9, 0, 0), (5, 32, 0, 0), (70, 64, 0, 0), (9, 64, 8, 0), (400, 128, 0, 0),
          (6, 128, 1, 0), (5, 136, 0, 0), (3, 200, 0, 3), (7, 255, 0, 0), (6, 264, 8, 8), (170, 512, 0, 0), (9, 1001, 6, 0),
          (700, 1000, 0, 0), (4, 4096, 0, 0), (3, 4104, 0, 1), (200, 2003, 3, 0), (2, 8192, 0, 0), (160, 8192, 0, 0), (3, 8191, 0, 0),
          (2, 8200, 0, 0), (3, 9001, 0, 5), (2, 16384, 0, 0), (2, 16392, 0, 0), (3, 20001, 1, 0)]


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_rms_forward(torch, v, rows, cols, pad, offset, dtype):  # noqa: F811
    _forward(torch, v, rows, cols, dtype, "float32", pad, offset)
    _forward(torch, v, rows, cols, dtype, dtype, pad, offset, residual=False)
    _forward(torch, v, rows, cols, dtype, "bfloat16", pad, offset, affine=False)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_rms_backward(torch, v, rows, cols, pad, offset, dtype):  # noqa: F811
    _backward(torch, v, rows, cols, dtype, "float32", pad, offset)
    _backward(torch, v, rows, cols, dtype, dtype, pad, offset, dsum=False)
    _backward(torch, v, rows, cols, dtype, "bfloat16", pad, offset, affine=False, dgamma=False)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(3001, 2003, 3, 0), (2500, 1001, 0, 1), (2000, 520, 8, 0), (700, 9000, 0, 0), (900, 4097, 0, 0),
                                                  (500, 9001, 0, 0), (310, 15001, 0, 0), (5000, 264, 1, 0)])
def test_rms_of_more_rows_than_stages(torch, v, rows, cols, pad, offset, dtype):  # noqa: F811
    """Every stage is filled again and again."""
    _forward(torch, v, rows, cols, dtype, "float32", pad, offset)
    _backward(torch, v, rows, cols, dtype, "float32", pad, offset)
    _forward(torch, v, rows, cols, dtype, "float32", pad, offset, residual=False, quant="e4m3", group=64 if cols % 2 else 0, with_y=False)
    _backward(torch, v, rows, cols, dtype, "float32", pad, offset, dsum=False)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols,opad,oskew", [(1500, 1001, 2, 3), (700, 4096, 1, 0), (320, 9001, 0, 1), (310, 13001, 4, 2), (2000, 130, 3, 1)])
def test_rms_of_many_rows_on_other_skews(torch, v, rows, cols, opad, oskew, dtype):  # noqa: F811
    """The outputs' rows on other skews than the inputs'."""
    _forward(torch, v, rows, cols, dtype, "float32", opad=opad, oskew=oskew)
    _backward(torch, v, rows, cols, dtype, "float32", opad=opad, oskew=oskew)
    _forward(torch, v, rows, cols, dtype, "float32", residual=False, quant="int8", opad=opad, oskew=oskew)
    _backward(torch, v, rows, cols, dtype, "float32", dsum=False, dgamma=False, opad=opad, oskew=oskew)


@pytest.mark.parametrize("cols", [1001, 9001, 20001])
def test_rms_in_place_beside_another_skew(torch, v, cols):  # noqa: F811
    """The sum in the place of x, y elsewhere on another skew."""
    g, rows = _rng(9), 330
    a, b = (g.standard_normal((rows, cols)) for _ in range(2))
    for offset, pad in ((3, 2), (5, 0), (0, 7)):
        x, r, s = Mat(torch, rows, cols, "float16", a, 0, 1), Mat(torch, rows, cols, "float16", b, 1, 2), Mat(torch, rows, cols, "float16", None, 0, 1)
        y, y2 = (Mat(torch, rows, cols, "float16", None, pad, offset) for _ in range(2))
        call = lambda s, y: v.vrcclRmsNormForward(x.ptr, r.ptr, None, s.ptr, y.ptr, None, rows, cols, "float16", "float32", ldx=x.ld,  # noqa: E731
                                                  ldr=r.ld, lds=s.ld, ldy=y.ld)
        call(s, y)
        call(x, y2)
        assert torch.equal(x.view, s.view) and torch.equal(y.view, y2.view) and x.intact() and y2.intact()


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 30, 0, 0), (50, 64, 0, 0), (9, 96, 0, 0), (30, 128, 16, 0), (5, 129, 0, 0),
                                                  (4, 1000, 0, 0), (7, 1001, 3, 0), (300, 512, 0, 0), (3, 4096, 0, 1),
                                                  (2, 8192, 0, 0), (2, 10000, 0, 0), (2, 9999, 2, 0)])
def test_rms_codes(torch, v, rows, cols, pad, offset, group, quant):  # noqa: F811
    for dtype in FLOATS:
        _forward(torch, v, rows, cols, dtype, "float32", pad, offset, quant=quant, group=group, with_y=dtype == "bfloat16",
                 residual=dtype != "float16")


@pytest.mark.parametrize("skew", range(8))
def test_rms_outputs_on_every_skew(torch, v, skew):  # noqa: F811
    for cols in (300, 8500):
        _forward(torch, v, 5, cols, "bfloat16", opad=3, oskew=skew)
        _backward(torch, v, 5, cols, "float16", pad=1, offset=2, opad=0, oskew=skew)
        _backward(torch, v, 5, cols, "float32", oskew=skew, opad=5)


def test_rms_of_zeros_and_extremes(torch, v):  # noqa: F811
    """A row of zeros has y 0 (eps alone under the root); tiny and huge rows are normed as they are."""
    for dtype in FLOATS:
        x = torch.zeros(3, 256, device="cuda", dtype=getattr(torch, dtype))
        y, codes, scales = torch.empty_like(x), torch.empty(3, 256, device="cuda", dtype=torch.int8), torch.empty(3, 2, device="cuda")
        v.vrcclRmsNormForward(x, None, None, None, y, None, 3, 256, dtype, dtype, codes=codes, scales=scales, group=128)
        assert (y == 0).all() and (codes == 0).all() and (scales == 2.0 ** -126).all()
    for scale in (1e-15, 1e-3, 1e15):
        _forward(torch, v, 4, 264, "float32", scale=scale, eps=0.0)
        _forward(torch, v, 4, 264, "bfloat16", scale=scale, eps=1e-30, quant="e4m3", group=64)


def test_rms_codes_show_what_is_not_finite(torch, v):  # noqa: F811
    """A NaN or infinity: the scales of its row's groups that it reaches are not finite, other rows are as they were."""
    g = _rng(4)
    base = torch.as_tensor(g.standard_normal((6, 512))).float().cuda()
    for quant, td in (("int8", torch.int8), ("e4m3", torch.float8_e4m3fn)):
        for group in (0, 64):
            for bad in (float("nan"), float("inf")):
                x = base.clone()
                x[2, 100] = bad
                codes, scales = torch.empty(6, 512, device="cuda", dtype=td), torch.empty(6, 8 if group else 1, device="cuda")
                v.vrcclRmsNormForward(x, None, None, None, None, None, 6, 512, "float32", "float32", codes=codes, scales=scales,
                                      quant=quant, group=group)
                fine = torch.isfinite(scales)
                assert not fine[2, 1 if group else 0] and fine[[0, 1, 3, 4, 5]].all()
                assert torch.isnan((codes.float() * scales.repeat_interleave(group or 512, 1))[2, 64 if group else 0:128]).all()


@pytest.mark.parametrize("dtype,cols,pad", [("bfloat16", 512, 0), ("bfloat16", 1001, 0), ("float32", 128, 0), ("float32", 9001, 3)])
def test_rms_in_place(torch, v, dtype, cols, pad):  # noqa: F811
    """sum and y in the place of x and residual, dx in that of each input."""
    g, rows = _rng(5), 400
    a, b, c = (g.standard_normal((rows, cols)) for _ in range(3))
    make = lambda q: Mat(torch, rows, cols, dtype, q, pad)  # noqa: E731
    s, y = make(None), make(None)
    x, r = make(a), make(b)
    args = (rows, cols, dtype, "float32")
    call = lambda x, r, s, y: v.vrcclRmsNormForward(x.ptr, r.ptr, None, s.ptr, y.ptr, None, *args, ldx=x.ld, ldr=r.ld, lds=s.ld, ldy=y.ld)  # noqa: E731
    call(x, r, s, y)
    for sum_over, y_over in ((0, 1), (1, 0), (0, None), (None, 0), (1, None), (None, 1)):
        m = [make(a), make(b)]
        s2, y2 = m[sum_over] if sum_over is not None else make(None), m[y_over] if y_over is not None else make(None)
        call(*m, s2, y2)
        assert torch.equal(s2.view, s.view) and torch.equal(y2.view, y.view) and s2.intact() and y2.intact()
    rstd = torch.rand(rows, device="cuda")
    ws = torch.empty(v.vrcclRmsNormWorkspace(rows, cols), device="cuda", dtype=torch.uint8)
    want, dg, dg2 = make(None), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    back = lambda d, e, s, o, q: v.vrcclRmsNormBackward(d.ptr, e.ptr, s.ptr, None, rstd, o.ptr, q, *args, ws, ws.numel(), lddy=d.ld,  # noqa: E731
                                                        lddsum=e.ld, lds=s.ld, lddx=o.ld)
    m = [make(q) for q in (a, b, c)]
    back(*m, want, dg)
    for over in range(3):
        m = [make(q) for q in (a, b, c)]
        back(*m, m[over], dg2)
        assert torch.equal(m[over].view, want.view) and torch.equal(dg, dg2) and m[over].intact()


def test_rms_gradient_against_differences(torch, v):  # noqa: F811
    """The backward pass against differences of the forward pass, in binary32 on smooth values."""
    g, rows, cols = _rng(6), 8, 96
    x, d, dy = (torch.as_tensor(g.standard_normal((rows, cols))).float().cuda() for _ in range(3))
    gamma = torch.rand(cols, device="cuda") + 0.5
    y, s, rstd, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty_like(x), torch.empty_like(gamma)
    ws = torch.empty(v.vrcclRmsNormWorkspace(rows, cols), device="cuda", dtype=torch.uint8)
    zero = torch.zeros_like(x)

    def f(a, w):
        v.vrcclRmsNormForward(a, zero, w, s, y, rstd, rows, cols, "float32", "float32")
        return (y.double() * dy.double()).sum().item()

    h = 1e-2
    f(x, gamma)
    v.vrcclRmsNormBackward(dy, None, s, gamma, rstd, dx, dg, rows, cols, "float32", "float32", ws, ws.numel())
    slope = (f(x + h * d, gamma) - f(x - h * d, gamma)) / (2 * h)
    # the third derivative along d times h^2 / 6 (some 10 |dy| |d| h^2), and the rounding of 768 values over 2 h
    tol = 10 * rows * cols * h * h / 6 + 768 ** 0.5 * 4 * EPS * 10 / h
    assert abs((dx.double() * d.double()).sum().item() - slope) <= tol
    e = torch.rand_like(gamma)
    slope = (f(x, gamma + h * e) - f(x, gamma - h * e)) / (2 * h)  # linear: rounding alone
    assert abs((dg.double() * e.double()).sum().item() - slope) <= 768 ** 0.5 * 4 * EPS * 10 / h + 1e-4


def test_rms_rows_beyond_32_bits(torch, v):  # noqa: F811
    ld, cols = (1 << 31) + 64, 520
    buf = torch.empty(2 * ld + cols + 1, device="cuda", dtype=torch.bfloat16)
    for shift in (0, 1):
        x = buf.as_strided((3, cols), (ld, 1), shift)
        x.copy_(torch.as_tensor(_rng(7).standard_normal((3, cols))))
        # the same rows close together, and on the same skew (on another one sums go in another order)
        flat = torch.empty(3 * 528 + 1, device="cuda", dtype=torch.bfloat16).as_strided((3, cols), (528, 1), shift)
        flat.copy_(x)
        y, want = torch.empty(3, cols, device="cuda", dtype=torch.bfloat16), torch.empty(3, cols, device="cuda", dtype=torch.bfloat16)
        r1, r2 = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
        v.vrcclRmsNormForward(x, None, None, None, y, r1, 3, cols, "bfloat16", "float32")
        v.vrcclRmsNormForward(flat, None, None, None, want, r2, 3, cols, "bfloat16", "float32")
        assert torch.equal(y, want) and torch.equal(r1, r2)
        v.vrcclRmsNormBackward(x, x, x, None, r1, y, None, 3, cols, "bfloat16", "float32")
        both = torch.empty_like(y)
        v.vrcclRmsNormBackward(flat, flat, flat, None, r1, both, None, 3, cols, "bfloat16", "float32")
        assert torch.equal(y, both)
        for rows in (x, flat):
            v.vrcclRmsNormBackward(rows, None, rows, None, r1, rows, None, 3, cols, "bfloat16", "float32")
        assert torch.equal(x, flat)


def test_rms_same_bits_in_graphs_and_on_streams(torch, v):  # noqa: F811
    rows, cols = 1000, 776
    g = torch.Generator("cuda").manual_seed(1)
    x, r, dy = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(3))
    s, y, dx = (torch.empty_like(x) for _ in range(3))
    rstd, gamma, dg = torch.empty(rows, device="cuda"), torch.rand(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(v.vrcclRmsNormWorkspace(rows, cols), device="cuda", dtype=torch.uint8)

    def step(stream=None):
        v.vrcclRmsNormForward(x, r, gamma, s, y, rstd, rows, cols, "bfloat16", "float32", stream=stream)
        v.vrcclRmsNormBackward(dy, y, s, gamma, rstd, dx, dg, rows, cols, "bfloat16", "float32", ws, ws.numel(), stream=stream)

    step()
    want = [t.clone() for t in (s, y, rstd, dx, dg)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for run in (graph.replay, lambda: step(side), graph.replay, step):
        for t in (s, y, rstd, dx, dg):
            t.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((s, y, rstd, dx, dg), want))
    assert v.vrcclReplicaGetAsyncError() == 0


def test_rms_of_no_rows(torch, v):  # noqa: F811
    dg = torch.ones(64, device="cuda")
    v.vrcclRmsNormBackward(None, None, None, None, None, None, dg, 0, 64, "float32", "float32")
    assert (dg == 0).all()
