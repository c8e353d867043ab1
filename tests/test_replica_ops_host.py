"""Host side of the replica's operators, no GPU needed: refusals before
anything is launched, workspace sizes, and the oracle's gradients against
differences."""
import ctypes

import numpy as np
import pytest

from oracle import replica as o

P, Z, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
A = [1 << 40 | i << 32 for i in range(16)]  # addresses 4 GiB apart, never dereferenced
I32, F32, BF16, F16, I8, I64 = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def lib():
    pytest.importorskip("torch")
    from ring_allreduce_reduction_gb300 import build
    build.build()
    from ring_allreduce_reduction_gb300 import vrccl
    return vrccl.LIB


def _call(fn, base, **change):
    args = dict(base, **change)
    assert list(args) == list(base)
    return fn(*args.values())


def test_norm_refusals(lib):
    fwd = dict(x=A[0], ldx=64, gamma=A[1], beta=A[2], y=A[3], ldy=64, mean=A[4], rstd=A[5], rows=4, cols=64, dtype=BF16,
               ptype=F32, eps=1e-5, stream=None)
    bad = [dict(x=None), dict(y=None), dict(x=A[0] + 1), dict(y=A[3] + 1), dict(gamma=A[1] + 2), dict(beta=A[2] + 2),
           dict(mean=A[4] + 2), dict(rstd=A[5] + 1), dict(ldx=63), dict(ldy=63), dict(dtype=I32), dict(dtype=7),
           dict(dtype=-1), dict(ptype=I8), dict(eps=-1.0), dict(eps=float("nan")), dict(cols=1 << 31),
           dict(rows=1 << 41), dict(y=A[0] + 64), dict(y=A[0], ldy=72), dict(ldx=1 << 41)]
    for change in bad:
        assert _call(lib.vrcclLayerNormForward, fwd, **change) == 1, change
    assert _call(lib.vrcclLayerNormForward, fwd, rows=0, x=None) == 0
    assert _call(lib.vrcclLayerNormForward, fwd, cols=0, x=None) == 0
    n = Z()
    assert lib.vrcclLayerNormWorkspace(4, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.vrcclLayerNormWorkspace(4, 64, None) == 1
    bwd = dict(dy=A[0], lddy=64, x=A[1], ldx=64, gamma=A[2], mean=A[3], rstd=A[4], dx=A[5], lddx=64, dgamma=A[6],
               dbeta=A[7], rows=4, cols=64, dtype=BF16, ptype=F32, ws=A[8], bytes=n.value, stream=None)
    bad = [dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(ws=None), dict(ws=A[8] + 4),
           dict(bytes=n.value - 1), dict(lddy=1), dict(ldx=1), dict(lddx=1), dict(dgamma=A[6] + 2), dict(dbeta=A[7] + 2),
           dict(dx=A[0] + 16), dict(dx=A[1], lddx=65), dict(dtype=I64), dict(ptype=7)]
    for change in bad:
        assert _call(lib.vrcclLayerNormBackward, bwd, **change) == 1, change
    assert _call(lib.vrcclLayerNormBackward, bwd, cols=0) == 0
    assert _call(lib.vrcclLayerNormBackward, bwd, rows=0, dgamma=None, dbeta=None) == 0


def test_linear_refusals(lib):
    fwd = dict(x=A[0], ldx=64, w=A[1], ldw=64, bias=A[2], r=A[3], ldr=32, y=A[4], ldy=32, z=A[5], ldz=32, rows=20, outs=32,
               ins=64, dtype=BF16, act=2, ws=A[6], bytes=1 << 20, stream=None)
    bad = [dict(x=None), dict(w=None), dict(y=None), dict(x=A[0] + 1), dict(bias=A[2] + 1), dict(r=A[3] + 1),
           dict(z=A[5] + 1), dict(ldx=63), dict(ldw=63), dict(ldr=31), dict(ldy=31), dict(ldz=31), dict(dtype=I32),
           dict(dtype=8), dict(act=5), dict(act=-1), dict(rows=1 << 31), dict(outs=1 << 31), dict(ins=1 << 31),
           dict(y=A[0]), dict(y=A[1]), dict(z=A[0]), dict(z=A[4]), dict(y=A[3], ldy=40), dict(y=A[2]), dict(ws=A[6] + 8),
           dict(ldx=65, bytes=16), dict(x=A[0] + 2, ws=None)]
    for change in bad:
        assert _call(lib.vrcclLinearForward, fwd, **change) == 1, change
    assert _call(lib.vrcclLinearForward, fwd, dtype=F32) == 2
    assert _call(lib.vrcclLinearForward, fwd, rows=0, x=None) == 0
    assert _call(lib.vrcclLinearForward, fwd, outs=0) == 0
    n = Z()
    assert lib.vrcclLinearWorkspace(1, 20, 32, 64, BF16, 2, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.vrcclLinearWorkspace(1, 20, 32, 64, F32, 2, ctypes.byref(n)) == 2
    assert lib.vrcclLinearWorkspace(0, 20, 32, 64, BF16, 9, ctypes.byref(n)) == 1
    assert lib.vrcclLinearWorkspace(0, 20, 32, 64, BF16, 0, None) == 1
    bwd = dict(dy=A[0], lddy=32, z=A[1], ldz=32, x=A[2], ldx=64, w=A[3], ldw=64, dx=A[4], lddx=64, dw=A[5], lddw=64,
               db=A[6], rows=20, outs=32, ins=64, dtype=BF16, act=2, ws=A[7], bytes=1 << 20, stream=None)
    bad = [dict(dy=None), dict(z=None), dict(x=None), dict(w=None), dict(dx=A[4] + 1), dict(dw=A[5] + 1), dict(db=A[6] + 1),
           dict(lddy=31), dict(ldz=31), dict(ldx=1), dict(ldw=1), dict(lddx=1), dict(lddw=1), dict(ws=None),
           dict(bytes=64), dict(dx=A[0]), dict(dw=A[3]), dict(dw=A[4]), dict(db=A[0]), dict(act=7), dict(dtype=I8),
           dict(ws=A[7] + 16)]
    for change in bad:
        assert _call(lib.vrcclLinearBackward, bwd, **change) == 1, change
    assert _call(lib.vrcclLinearBackward, bwd, dtype=F32) == 2
    assert lib.vrcclReplicaGetAsyncError(None) == 1


def test_distill_refusals(lib):
    fwd = dict(s=A[0], ldl=100, t=A[1], ldt=8, idx=A[2], ldi=8, loss=A[3], stats=A[4], rows=4, vocab=100, k=8, dtype=BF16,
               ttype=F32, itype=I64, T=1.0, stream=None)
    bad = [dict(s=None), dict(t=None), dict(idx=None), dict(loss=None), dict(s=A[0] + 1), dict(t=A[1] + 2),
           dict(idx=A[2] + 4), dict(loss=A[3] + 2), dict(stats=A[4] + 4), dict(ldl=99), dict(ldt=7), dict(ldi=7),
           dict(k=1025, ldt=2000, ldi=2000), dict(dtype=I32), dict(ttype=I64), dict(itype=F32), dict(T=0.0), dict(T=-1.0),
           dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-39), dict(rows=1 << 31), dict(vocab=1 << 31)]
    for change in bad:
        assert _call(lib.vrcclDistillForward, fwd, **change) == 1, change
    assert _call(lib.vrcclDistillForward, fwd, rows=0) == 0
    bwd = dict(s=A[0], ldl=100, t=A[1], ldt=8, idx=A[2], ldi=8, stats=A[3], dloss=A[4], stride=1, ds=A[5], ldd=100, rows=4,
               vocab=100, k=8, dtype=BF16, ttype=F32, itype=I64, T=1.0, stream=None)
    bad = [dict(s=None), dict(ds=None), dict(stats=None), dict(dloss=None), dict(stats=A[3] + 4), dict(dloss=A[4] + 2),
           dict(ds=A[5] + 1), dict(ldd=99), dict(ds=A[0] + 2), dict(ds=A[0], ldd=101), dict(k=2000, ldt=2000, ldi=2000),
           dict(stride=1 << 41)]
    for change in bad:
        assert _call(lib.vrcclDistillBackward, bwd, **change) == 1, change
    assert _call(lib.vrcclDistillBackward, bwd, rows=0) == 0
    assert _call(lib.vrcclDistillBackward, bwd, vocab=0) == 0


def test_outputs_that_overlap_are_refused(lib):
    """An output may not touch an input, another output or the workspace, other than in place as documented."""
    norm = dict(x=A[0], ldx=64, gamma=A[1], beta=A[2], y=A[3], ldy=64, mean=A[4], rstd=A[5], rows=4, cols=64, dtype=BF16,
                ptype=F32, eps=1e-5, stream=None)
    for change in (dict(mean=A[3] + 64), dict(rstd=A[4] + 8), dict(y=A[1]), dict(y=A[2] + 128), dict(mean=A[0] + 8),
                   dict(x=A[3], ldx=72), dict(rstd=A[1])):
        assert _call(lib.vrcclLayerNormForward, norm, **change) == 1, change
    back = dict(dy=A[0], lddy=64, x=A[1], ldx=64, gamma=A[2], mean=A[3], rstd=A[4], dx=A[5], lddx=64, dgamma=A[6],
                dbeta=A[7], rows=4, cols=64, dtype=BF16, ptype=F32, ws=A[8], bytes=1 << 20, stream=None)
    for change in (dict(ws=A[5]), dict(ws=A[0]), dict(dgamma=A[1] + 4), dict(dbeta=A[6] + 16), dict(dx=A[3]), dict(dgamma=A[2]),
                   dict(dbeta=A[8] + 64)):
        assert _call(lib.vrcclLayerNormBackward, back, **change) == 1, change
    lin = dict(x=A[0], ldx=64, w=A[1], ldw=64, bias=A[2], r=A[3], ldr=32, y=A[4], ldy=32, z=A[5], ldz=32, rows=20, outs=32,
               ins=64, dtype=BF16, act=2, ws=A[6], bytes=1 << 20, stream=None)
    for change in (dict(z=A[3]), dict(ws=A[4]), dict(ws=A[0]), dict(ws=A[3]), dict(z=A[2])):
        assert _call(lib.vrcclLinearForward, lin, **change) == 1, change
    grad = dict(dy=A[0], lddy=32, z=A[1], ldz=32, x=A[2], ldx=64, w=A[3], ldw=64, dx=A[4], lddx=64, dw=A[5], lddw=64,
                db=A[6], rows=20, outs=32, ins=64, dtype=BF16, act=2, ws=A[7], bytes=1 << 20, stream=None)
    for change in (dict(ws=A[4]), dict(ws=A[1]), dict(db=A[5] + 2), dict(dx=A[1]), dict(db=A[2])):
        assert _call(lib.vrcclLinearBackward, grad, **change) == 1, change
    dis = dict(s=A[0], ldl=100, t=A[1], ldt=8, idx=A[2], ldi=8, loss=A[3], stats=A[4], rows=4, vocab=100, k=8, dtype=BF16,
               ttype=F32, itype=I64, T=1.0, stream=None)
    for change in (dict(loss=A[0] + 4), dict(stats=A[1]), dict(loss=A[4] + 8), dict(stats=A[2])):
        assert _call(lib.vrcclDistillForward, dis, **change) == 1, change
    dback = dict(s=A[0], ldl=100, t=A[1], ldt=8, idx=A[2], ldi=8, stats=A[3], dloss=A[4], stride=1, ds=A[5], ldd=100, rows=4,
                 vocab=100, k=8, dtype=BF16, ttype=F32, itype=I64, T=1.0, stream=None)
    for change in (dict(ds=A[1]), dict(ds=A[2]), dict(ds=A[3]), dict(ds=A[4])):
        assert _call(lib.vrcclDistillBackward, dback, **change) == 1, change


def test_extents_beyond_64_bits_are_refused(lib):
    """Rows times row stride must stay addressable; a temperature's square and reciprocal normal numbers."""
    norm = dict(x=A[0], ldx=1 << 39, gamma=None, beta=None, y=A[3], ldy=64, mean=None, rstd=None, rows=1 << 30, cols=64,
                dtype=BF16, ptype=F32, eps=1e-5, stream=None)
    assert _call(lib.vrcclLayerNormForward, norm) == 1
    dis = dict(s=A[0], ldl=100, t=A[1], ldt=8, idx=A[2], ldi=8, loss=A[3], stats=A[4], rows=4, vocab=100, k=8, dtype=BF16,
               ttype=F32, itype=I64, T=1.0, stream=None)
    for change in (dict(T=1e-19), dict(T=1e19), dict(ldl=1 << 39, rows=1 << 20), dict(ldi=1 << 39, rows=1 << 20)):
        assert _call(lib.vrcclDistillForward, dis, **change) == 1, change


def _along(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_oracle_gradients_against_differences():
    g = np.random.default_rng(1)
    x, dy = g.standard_normal((5, 12)), g.standard_normal((5, 12))
    gamma, beta = g.standard_normal(12), g.standard_normal(12)
    _, mean, rstd = o.norm_forward(x, gamma, beta, 1e-5)
    dx, dg, db = o.norm_backward(dy, x, gamma, mean, rstd)
    for grad, at in ((dx, 0), (dg, 1), (db, 2)):
        d = g.standard_normal(grad.shape)
        args = [x, gamma, beta]
        f = lambda a: (dy * o.norm_forward(*[a if i == at else args[i] for i in range(3)], 1e-5)[0]).sum()  # noqa: E731
        assert abs((grad * d).sum() - _along(f, args[at], d)) < 1e-7
    w, b, r, dy = g.standard_normal((7, 12)), g.standard_normal(7), g.standard_normal((5, 7)), g.standard_normal((5, 7))
    for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
        _, z = o.linear_forward(x, w, b, r, act)
        for at, grad in enumerate(o.linear_backward(dy, z, x, w, act)):
            d = g.standard_normal(grad.shape)
            args = [x, w, b]
            f = lambda a: (dy * o.linear_forward(*[a if i == at else args[i] for i in range(3)], r, act)[0]).sum()  # noqa: E731
            assert abs((grad * d).sum() - _along(f, args[at], d)) < 1e-6
    s, t, idx = g.standard_normal((4, 30)), g.standard_normal((4, 6)), g.integers(0, 30, (4, 6))
    idx[1] = -1
    idx[2, 3:] = idx[2, 0]
    dl = g.standard_normal(4)
    grad, d = o.distill_backward(s, t, idx, dl, 2.0), g.standard_normal((4, 30))
    assert abs((grad * d).sum() - _along(lambda a: (dl * o.distill_forward(a, t, idx, 2.0)[0]).sum(), s, d)) < 1e-7
