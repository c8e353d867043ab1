"""Host side of the replica's dropout, RMS norm and token log probabilities, no
GPU needed: refusals before anything is launched, workspace sizes, the
binding's checks, and the oracle's gradients against differences."""
import ctypes

import numpy as np
import pytest

from oracle import replica as o
from test_replica_binding import NoLibrary, v  # noqa: F401
from test_replica_ops_host import A, BF16, F16, F32, I32, I64, I8, Z, _along, _call, lib  # noqa: F401


def test_dropout_refusals(lib):  # noqa: F811
    fwd = dict(x=A[0], ldx=64, r=A[1], ldr=64, y=A[2], ldy=64, rows=4, cols=64, dtype=BF16, p=0.1, seed=A[3], offset=1, first=0,
               stream=None)
    bad = [dict(x=None), dict(y=None), dict(seed=None), dict(x=A[0] + 1), dict(r=A[1] + 1), dict(y=A[2] + 1), dict(seed=A[3] + 4),
           dict(ldx=63), dict(ldr=63), dict(ldy=63), dict(dtype=I32), dict(dtype=I8), dict(dtype=9), dict(dtype=-1), dict(p=-0.1),
           dict(p=1.5), dict(p=float("nan")), dict(rows=1 << 41), dict(cols=1 << 31), dict(ldx=1 << 41), dict(first=1 << 40),
           dict(y=A[0] + 64), dict(y=A[0], ldy=72), dict(y=A[1], ldr=72), dict(y=A[3]), dict(seed=A[2] + 8),
           dict(ldx=1 << 39, rows=1 << 30)]
    for change in bad:
        assert _call(lib.vrcclDropoutForward, dict(fwd, p=ctypes.c_float(fwd["p"])),
                     **{k: ctypes.c_float(x) if k == "p" else x for k, x in change.items()}) == 1, change
    assert _call(lib.vrcclDropoutForward, fwd, rows=0, x=None) == 0
    assert _call(lib.vrcclDropoutForward, fwd, cols=0, y=None) == 0
    bwd = dict(dy=A[0], lddy=64, dx=A[2], lddx=64, rows=4, cols=64, dtype=F16, p=0.1, seed=A[3], offset=1, first=0, stream=None)
    for change in (dict(dy=None), dict(dx=None), dict(seed=None), dict(lddy=1), dict(lddx=1), dict(dx=A[0] + 2), dict(p=2.0),
                   dict(dx=A[0], lddx=65), dict(dtype=I64)):
        assert _call(lib.vrcclDropoutBackward, bwd, **change) == 1, change
    assert _call(lib.vrcclDropoutBackward, bwd, rows=0) == 0


RMS = dict(x=A[0], ldx=64, r=A[1], ldr=64, gamma=A[2], sum=A[3], lds=64, y=A[4], ldy=64, codes=None, ldc=0, scales=None, ldsc=0,
           rstd=A[5], rows=4, cols=64, dtype=BF16, ptype=F32, quant=0, group=0, eps=1e-5, stream=None)
CODES = dict(RMS, codes=A[6], ldc=64, scales=A[7], ldsc=2, group=32)


def test_rms_refusals(lib):  # noqa: F811
    bad = [dict(x=None), dict(y=None), dict(x=A[0] + 1), dict(r=A[1] + 1), dict(gamma=A[2] + 2), dict(sum=A[3] + 1),
           dict(y=A[4] + 1), dict(rstd=A[5] + 2), dict(ldx=63), dict(ldr=63), dict(lds=63), dict(ldy=63), dict(dtype=I32),
           dict(dtype=7), dict(ptype=I8), dict(eps=-1.0), dict(eps=float("nan")), dict(cols=1 << 31), dict(rows=1 << 41),
           dict(y=A[0] + 64), dict(y=A[0], ldy=72), dict(sum=A[0] + 64), dict(sum=A[1], lds=72), dict(y=A[3]),
           dict(y=A[0], sum=A[0]), dict(y=A[2]), dict(sum=A[2]), dict(rstd=A[3] + 8), dict(rstd=A[0]), dict(rstd=A[1]), dict(rstd=A[4])]
    for change in bad:
        assert _call(lib.vrcclRmsNormForward, RMS, **change) == 1, change
    bad = [dict(quant=2), dict(quant=-1), dict(group=1), dict(group=16), dict(group=96), dict(group=256), dict(ldc=63),
           dict(scales=None), dict(scales=A[7] + 2), dict(ldsc=1), dict(codes=A[0]), dict(codes=A[3] + 1), dict(codes=A[4] + 1),
           dict(scales=A[6]), dict(scales=A[0]), dict(scales=A[5]), dict(rstd=A[6] + 4), dict(codes=A[2])]
    for change in bad:
        assert _call(lib.vrcclRmsNormForward, CODES, **change) == 1, change
    assert _call(lib.vrcclRmsNormForward, RMS, rows=0, x=None) == 0
    assert _call(lib.vrcclRmsNormForward, RMS, cols=0, x=None) == 0
    n = Z()
    assert lib.vrcclRmsNormWorkspace(4, 64, ctypes.byref(n)) == 0 and n.value >= 64 * 4
    assert lib.vrcclRmsNormWorkspace(4, 64, None) == 1
    assert lib.vrcclRmsNormWorkspace(4, 1 << 31, ctypes.byref(n)) == 1
    assert lib.vrcclRmsNormWorkspace(4, 64, ctypes.byref(n)) == 0
    bwd = dict(dy=A[0], lddy=64, dsum=A[1], ldds=64, s=A[2], lds=64, gamma=A[3], rstd=A[4], dx=A[5], lddx=64, dgamma=A[6], rows=4,
               cols=64, dtype=BF16, ptype=F32, ws=A[7], bytes=n.value, stream=None)
    bad = [dict(dy=None), dict(s=None), dict(dx=None), dict(rstd=None), dict(ws=None), dict(ws=A[7] + 4), dict(bytes=n.value - 1),
           dict(lddy=1), dict(ldds=1), dict(lds=1), dict(lddx=1), dict(dgamma=A[6] + 2), dict(dsum=A[1] + 1), dict(dx=A[0] + 16),
           dict(dx=A[2], lddx=65), dict(dx=A[1] + 2), dict(dtype=I64), dict(ptype=7), dict(ws=A[5]), dict(ws=A[0]), dict(ws=A[1]),
           dict(dgamma=A[2] + 4), dict(dgamma=A[3]), dict(dgamma=A[7] + 64), dict(dx=A[4]), dict(dx=A[3])]
    for change in bad:
        assert _call(lib.vrcclRmsNormBackward, bwd, **change) == 1, change
    assert _call(lib.vrcclRmsNormBackward, bwd, cols=0) == 0
    assert _call(lib.vrcclRmsNormBackward, bwd, rows=0, dgamma=None) == 0


def test_logprob_refusals(lib):  # noqa: F811
    fwd = dict(s=A[0], ldl=100, token=A[1], logprob=A[2], entropy=A[3], stats=A[4], top=A[5], ldt=8, index=A[6], ldi=8, rows=4,
               vocab=100, k=8, dtype=BF16, ttype=I64, T=1.0, stream=None)
    bad = [dict(s=None), dict(token=None), dict(top=None), dict(index=None), dict(s=A[0] + 1), dict(token=A[1] + 4),
           dict(logprob=A[2] + 2), dict(entropy=A[3] + 1), dict(stats=A[4] + 4), dict(top=A[5] + 2), dict(index=A[6] + 1),
           dict(ldl=99), dict(ldt=7), dict(ldi=7), dict(k=33, ldt=40, ldi=40), dict(dtype=I32), dict(ttype=F32), dict(T=0.0),
           dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-19), dict(T=1e19), dict(rows=1 << 31),
           dict(vocab=1 << 31), dict(ldl=1 << 39, rows=1 << 20), dict(logprob=A[0]), dict(entropy=A[1]), dict(stats=A[0] + 8),
           dict(top=A[6]), dict(index=A[4]), dict(entropy=A[2] + 4), dict(logprob=A[5] + 4)]
    for change in bad:
        assert _call(lib.vrcclLogProbForward, fwd, **change) == 1, change
    assert _call(lib.vrcclLogProbForward, fwd, rows=0) == 0
    bwd = dict(s=A[0], ldl=100, token=A[1], stats=A[2], entropy=A[3], dl=A[4], dls=1, dh=A[5], dhs=1, ds=A[6], ldd=100, rows=4,
               vocab=100, dtype=BF16, ttype=I64, T=1.0, stream=None)
    bad = [dict(s=None), dict(ds=None), dict(stats=None), dict(token=None), dict(entropy=None), dict(dl=None, dh=None),
           dict(stats=A[2] + 4), dict(dl=A[4] + 2), dict(dh=A[5] + 2), dict(ds=A[6] + 1), dict(ldd=99), dict(ds=A[0] + 2),
           dict(ds=A[0], ldd=101), dict(dls=1 << 41), dict(dhs=1 << 41), dict(ds=A[1]), dict(ds=A[2]), dict(ds=A[3]),
           dict(ds=A[4]), dict(ds=A[5])]
    for change in bad:
        assert _call(lib.vrcclLogProbBackward, bwd, **change) == 1, change
    assert _call(lib.vrcclLogProbBackward, bwd, rows=0) == 0
    assert _call(lib.vrcclLogProbBackward, bwd, vocab=0) == 0


def test_rms_workspace_covers_the_call(lib):  # noqa: F811
    """The query says whole rows of binary32 sums, one at least and no more than the rows."""
    n = Z()
    for cols in (1, 64, 128, 129, 1001, 4096, 8192, 8193, 16384, 16385, 50000):
        for rows in (1, 2, 100, 152, 1000, 5000, 100000):
            assert lib.vrcclRmsNormWorkspace(rows, cols, ctypes.byref(n)) == 0
            assert cols * 4 <= n.value <= rows * cols * 4 and n.value % (cols * 4) == 0


def test_binding_refusals(v, monkeypatch):  # noqa: F811
    """Tensors that do not fit: before the library is called."""
    import torch
    monkeypatch.setattr(v, "_lib", NoLibrary())
    x, seed = torch.zeros(4, 64), torch.zeros(1, dtype=torch.int32)
    drop = dict(x=4096, residual=None, y=8192, rows=4, cols=64, dtype="float32", p=0.1, seed=12288)
    rms = dict(x=4096, residual=None, gamma=None, sum=None, y=8192, rstd=None, rows=4, cols=64, dtype="bfloat16", ptype="float32")
    log = dict(logits=4096, token=8192, logprob=12288, entropy=None, stats=None, top=None, top_index=None, rows=4, vocab=64, k=0,
               dtype="float32", token_dtype="int64")
    for fn, base, change, why in (
            (v.vrcclDropoutForward, drop, dict(x=x), "cpu"),
            (v.vrcclDropoutForward, drop, dict(seed=seed), "int32"),
            (v.vrcclDropoutForward, drop, dict(residual=x.half()), "float16"),
            (v.vrcclRmsNormForward, rms, dict(residual=x), "float32"),
            (v.vrcclRmsNormForward, rms, dict(codes=x.to(torch.uint8), scales=4096), "uint8"),
            (v.vrcclRmsNormForward, rms, dict(codes=x.to(torch.int8), scales=4096, quant="e4m3"), "int8"),
            (v.vrcclRmsNormForward, rms, dict(codes=4096, scales=x.double()), "float64"),
            (v.vrcclRmsNormForward, rms, dict(codes=4096, scales=4096, quant="int4"), "int4"),
            (v.vrcclLogProbForward, log, dict(token=torch.zeros(4, dtype=torch.int32)), "int32"),
            (v.vrcclLogProbForward, log, dict(logprob=torch.zeros(4)), "cpu"),
            (v.vrcclLogProbForward, log, dict(k=2, top=torch.zeros(4, 2).half(), top_index=4096), "float16")):
        with pytest.raises(ValueError, match=why):
            fn(**dict(base, **change))


def test_oracle_gradients_against_differences():
    g = np.random.default_rng(2)
    s, gamma, dy, dsum = g.standard_normal((5, 12)), g.standard_normal(12), g.standard_normal((5, 12)), g.standard_normal((5, 12))
    _, rstd = o.rms_forward(s, gamma, 1e-5)
    for at, grad in enumerate(o.rms_backward(dy, dsum, s, gamma, rstd)):
        d, args = g.standard_normal(grad.shape), [s, gamma]
        f = lambda a: ((dy * o.rms_forward(*[a if i == at else args[i] for i in range(2)], 1e-5)[0]).sum()  # noqa: E731
                       + (dsum * (a if at == 0 else s)).sum())
        assert abs((grad * d).sum() - _along(f, args[at], d)) < 1e-7
    x, token = g.standard_normal((5, 30)) * 2, np.array([3, 29, -1, 0, 30])
    x[3, 5:9] = -np.inf
    dl, dh = g.standard_normal(5), g.standard_normal(5)
    grad, d = o.logprob_backward(x, token, dl, dh, 0.7), g.standard_normal((5, 30))
    f = lambda a: sum((w * y).sum() for w, y in zip((dl, dh), o.logprob_forward(a, token, 2, 0.7)))  # noqa: E731
    assert abs((grad * d).sum() - _along(f, x, d)) < 1e-7
    x, r = g.standard_normal((3, 20)), g.standard_normal((3, 20))
    kept, scale = o.dropout_mask(3, 20, 0.3, 5, 6, 7)
    d = g.standard_normal((3, 20))
    f = lambda a: (dy[:3, :1] * o.dropout(a, r, 0.3, 5, 6, 7)).sum()  # noqa: E731
    assert abs((np.where(kept, dy[:3, :1] * scale, 0) * d).sum() - _along(f, x, d)) < 1e-8


def test_oracle_mask_is_of_rows_and_expectation():
    """Rows of a mask do not depend on where a call begins; the kept share is the probability's."""
    whole, scale = o.dropout_mask(24, 130, 0.25, 9, 3, 100)
    part, _ = o.dropout_mask(4, 130, 0.25, 9, 3, 110)
    assert np.array_equal(whole[10:14], part) and scale == 65536 / (65536 - 16384)
    n = whole.size
    assert abs(whole.mean() - 0.75) < 5 * np.sqrt(0.75 * 0.25 / n)
    assert not np.array_equal(whole, o.dropout_mask(24, 130, 0.25, 9, 4, 100)[0])
