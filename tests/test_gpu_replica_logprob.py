"""Token log probabilities on the GPU against their definition in 64 bits
(oracle/replica.py): values, entropy, the order of the alternatives, gradients
against the formula and against differences, masks, padding, ties, strides,
alignment, in place. Helpers and U, EPS, TINY as in test_gpu_replica_ops.py.

Tolerances. x = (s - max) / T in units of log 2 carries three roundings, 2^x an
error of 4 EPS of its own, so a term is off by at most (2.1 |x| + 4) EPS of
itself; a sum adds one EPS for each addition that a term goes through: a
thread's share (the vocabulary over 128 threads at least) and the joins (64).
The entropy's second sum weighs the same errors by |x|."""
import numpy as np
import pytest

from oracle import replica as o
from test_gpu_replica_ops import EPS, FLOATS, TINY, U, Mat, _close, _host, _rng, torch, v  # noqa: F401

pytestmark = pytest.mark.gpu


def _errors(s, T):
    """(error of log sum exp, error of the entropy) of one row of finite largest logit."""
    with np.errstate(invalid="ignore"):
        x = (s - s.max()) / T
        e = np.exp(x)
        l = e.sum()
        seen = np.where(e > 0, np.abs(x), 0)
        n = s.size / 128 + 64
        el = (n + ((3 * seen + 4) * e).sum() / l) * EPS
        ew = (((n + 8 + 3 * seen) * seen * e).sum() / l) * EPS + el * (seen * e).sum() / l
    return el + 2 * EPS * abs(np.log(l)), ew + el + 4 * EPS * abs(np.log(l))


def _inputs(torch, rows, vocab, dtype, pad=0, offset=0, padding=0.2, scale=2.5, seed=1, itype="int64"):  # noqa: F811
    g = _rng(seed)
    s = Mat(torch, rows, vocab, dtype, scale * g.standard_normal((rows, vocab)), pad, offset)
    token = g.integers(0, vocab, rows)
    lost = g.random(rows) < padding
    token[lost] = g.choice([-1, -100, vocab, vocab + 5], lost.sum())
    return s, token, torch.as_tensor(token).to("cuda", getattr(torch, itype))


def _forward(torch, v, s, token, k, dtype, T=1.0, itype="int64", given=None):  # noqa: F811
    rows, vocab = s.rows, s.cols
    dev = torch.as_tensor(token).to("cuda", getattr(torch, itype)) if token is not None else None
    logprob = torch.full((rows,), 7.0, device="cuda") if token is not None else None
    entropy, stats = torch.full((rows,), 7.0, device="cuda"), torch.full((rows, 2), 7.0, device="cuda")
    top = torch.full((rows, k + 1), 7.0, device="cuda") if k else None
    index = torch.full((rows, k + 2), 7, device="cuda", dtype=torch.int32) if k else None
    v.vrcclLogProbForward(s.ptr, dev, logprob, entropy, stats, top, index, rows, vocab, k, dtype, itype, T, ldl=s.ld, ldt=k + 1,
                          ldi=k + 2)
    S = s.get()
    wl, we, ws, wt, wi = o.logprob_forward(S, token, k, T)
    # outputs are binary32: what lies beyond its largest value (a float's lowest over a temperature below one) is infinite
    wl, wt = (np.where(q < -float(np.finfo(np.float32).max), -np.inf, q) for q in (wl, wt))
    tl, te = np.zeros(rows), np.zeros(rows)
    for r in range(rows):
        if np.isfinite(S[r].max()):
            tl[r], te[r] = _errors(S[r], T)
    _close(_host(entropy), we, te, "entropy")
    _close(_host(stats)[:, 0], ws[:, 0], 0, "largest")
    _close(_host(stats)[:, 1], ws[:, 1], tl, "log sum")
    with np.errstate(invalid="ignore"):
        far = lambda q: 4 * EPS * (np.abs(q) + np.abs(ws[:, 1]).reshape(-1, *[1] * (q.ndim - 1)))  # noqa: E731
        if token is not None:
            _close(_host(logprob), wl, tl + far(wl), "logprob")
        if k:
            assert np.array_equal(index[:, :k].cpu().numpy(), wi), "alternatives"
            _close(_host(top[:, :k]), wt, tl[:, None] + far(wt), "their log probabilities")
            assert (top[:, k:] == 7).all() and (index[:, k:] == 7).all()
    assert s.intact()
    return dev, entropy, stats


def _backward(torch, v, s, token, dev, entropy, stats, dtype, T=1.0, pad=0, oskew=0, use=(True, True), in_place=False, itype="int64",  # noqa: F811
              seed=3):
    g, rows, vocab = _rng(seed), s.rows, s.cols
    S = s.get()
    dl, dh = (torch.as_tensor(g.standard_normal(rows)).float().cuda() for _ in range(2))
    use = (use[0] and token is not None, use[1])
    DL, DH = _host(dl) * use[0], _host(dh) * use[1]
    out = s if in_place else Mat(torch, rows, vocab, dtype, None, pad, oskew)
    v.vrcclLogProbBackward(s.ptr, dev, stats, entropy if use[1] else None, dl if use[0] else None, dh if use[1] else None, out.ptr,
                           rows, vocab, dtype, itype, T, ldl=s.ld, ldd=out.ld)
    want = o.logprob_backward(S, token, DL, DH, T)
    tol = np.zeros_like(want)
    for r in range(rows):
        if not np.isfinite(S[r].max()):
            continue
        el, eh = _errors(S[r], T)
        with np.errstate(invalid="ignore"):
            logq = o._logq(S[r], T)
            q = np.exp(logq)
            known, h = np.where(q > 0, -logq, 0), -np.sum(q * np.where(q > 0, logq, 0))
        ll = abs(np.log(np.exp((S[r] - S[r].max()) / T).sum()))
        part = q * (abs(DL[r]) + abs(DH[r]) * (known + h)) / T
        # the share's own error (its exponent's roundings, the saved sum's) and the factor's
        tol[r] = part * (el + EPS * (16 + 4 * known + 4 * ll)) + q * abs(DH[r]) * (eh + el) / T
    tol += U[dtype] * 1.01 * np.abs(want) + 4 * EPS * np.abs(DL[:, None]) / T * (np.arange(vocab) == (token[:, None] if token is not None else -1))
    _close(out.get(), want, tol + TINY[dtype], "dlogits")
    assert out.intact()


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,vocab,k,pad,offset", [(1, 1, 1, 0, 0), (3, 2, 5, 0, 1), (5, 7, 3, 0, 0), (4, 8, 8, 0, 0), (9, 31, 32, 2, 3),
                                                     (6, 1000, 5, 0, 0), (5, 1001, 20, 3, 1), (40, 4099, 1, 0, 0), (3, 16384, 32, 8, 0),
                                                     (700, 2049, 7, 0, 0), (2, 50001, 20, 0, 7), (3, 131072, 20, 0, 0),
                                                     (1, 131075, 32, 0, 5), (330, 33000, 0, 0, 0)])
def test_logprob(torch, v, rows, vocab, k, pad, offset, dtype):  # noqa: F811
    for T, itype, padding in ((1.0, "int64", 0.2), (0.7, "int32", 0.0)):
        s, token, _ = _inputs(torch, rows, vocab, dtype, pad, offset, padding)
        dev, entropy, stats = _forward(torch, v, s, token, k, dtype, T, itype)
        if rows * vocab <= 2e6:
            _backward(torch, v, s, token, dev, entropy, stats, dtype, T, pad, offset, itype=itype)
            _backward(torch, v, s, token, dev, entropy, stats, dtype, T, 1, 3, (True, False), itype=itype)
            _backward(torch, v, s, token, dev, entropy, stats, dtype, T, in_place=True, use=(False, True), itype=itype)


def test_logprob_without_tokens(torch, v):  # noqa: F811
    """Alternatives and entropy alone, as for the next token; the entropy's gradient."""
    s, _, _ = _inputs(torch, 6, 3001, "bfloat16")
    _, entropy, stats = _forward(torch, v, s, None, 12, "bfloat16", 1.3)
    _backward(torch, v, s, None, None, entropy, stats, "bfloat16", 1.3)


@pytest.mark.parametrize("dtype", FLOATS)
def test_logprob_masked(torch, v, dtype):  # noqa: F811
    """-inf and the type's lowest value, rows of nothing else, one entry left, padding that holds NaN."""
    low = float(torch.finfo(getattr(torch, dtype)).min)
    for vocab in (64, 1003, 40000):
        s, token, _ = _inputs(torch, 9, vocab, dtype, padding=0)
        a = s.view
        a[0, ::2] = -float("inf")
        a[1, 1:] = low
        a[2, :] = -float("inf")
        a[3, :] = -float("inf")
        a[3, vocab // 2] = -2.0
        a[4, :] = low
        a[5, : vocab // 3] = low
        a[5, vocab // 3: vocab // 2] = -float("inf")
        a[6, :] = float("nan")
        a[7, 3:] = -float("inf")
        token[3], token[6], token[7] = vocab // 2, -1, vocab - 1
        for T in (1.0, 0.5):
            dev, entropy, stats = _forward(torch, v, s, token, 9, dtype, T)
            _backward(torch, v, s, token, dev, entropy, stats, dtype, T)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_logprob_of_huge_logits(torch, v, dtype):  # noqa: F811
    """Logits whose differences are all there is: offsets at which a product with 1 / T keeps no fraction."""
    for vocab, T in ((300, 1.0), (9000, 0.5)):
        s, token, _ = _inputs(torch, 8, vocab, dtype, padding=0)
        for r, big in enumerate((2e5, -3e7, 1e8, 5e9, -1e12, 1e30, -1e37, 0)):
            s.view[r] = (s.view[r].double() * max(1.0, abs(big) * 2.0 ** -8) + big).to(s.view.dtype)
        s.view[7, ::3] *= 1e20
        dev, entropy, stats = _forward(torch, v, s, token, 6, dtype, T)
        _backward(torch, v, s, token, dev, entropy, stats, dtype, T)


def test_logprob_of_rows_that_are_not_finite(torch, v):  # noqa: F811
    """A NaN or +inf makes the row's values NaN; the alternatives keep their order, a NaN first."""
    for vocab in (500, 20001):
        s, token, _ = _inputs(torch, 5, vocab, "float32", padding=0)
        s.view[1, 77] = float("nan")
        s.view[2, 5] = float("inf")
        s.view[2, 499] = float("inf")
        s.view[3, 9] = float("inf")
        s.view[3, 300] = float("nan")
        s.view[3, 200] = float("nan")
        top, index = torch.empty(5, 4, device="cuda"), torch.empty(5, 4, device="cuda", dtype=torch.int32)
        lp, h, st = torch.empty(5, device="cuda"), torch.empty(5, device="cuda"), torch.empty(5, 2, device="cuda")
        dev = torch.as_tensor(token).cuda()
        v.vrcclLogProbForward(s.ptr, dev, lp, h, st, top, index, 5, vocab, 4, "float32", "int64")
        bad = np.array([False, True, True, True, False])
        for t in (lp, h, top[:, 1]):
            assert np.array_equal(np.isnan(_host(t)), bad)
        _, _, _, _, wi = o.logprob_forward(s.get(), token, 4, 1.0)
        assert np.array_equal(index.cpu().numpy(), wi)
        d = torch.empty(5, vocab, device="cuda")
        v.vrcclLogProbBackward(s.ptr, dev, st, h, torch.ones(5, device="cuda"), torch.ones(5, device="cuda"), d, 5, vocab, "float32", "int64")
        assert np.array_equal(np.isnan(_host(d)).all(1), bad) and np.array_equal(np.isnan(_host(d)).any(1), bad)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("vocab", [100, 5000, 66000])
def test_alternatives_of_awkward_rows(torch, v, vocab, dtype):  # noqa: F811
    """Ties everywhere, zeros of both signs, rising and falling rows, all of the largest in one thread's share."""
    n = np.arange(vocab)
    rows = [np.zeros(vocab), np.where(n % 3 == 0, 0.0, -0.0), np.minimum(n, 2000) / 16, -np.minimum(n, 2000) / 16, (n % 7).astype(float),
            np.where(n % 4096 < 8, 3 + (n % 8) / 8, -1), np.where(n % 1024 < 8, 3.0, -1.0), np.where(n > vocab - 30, 2.0, 1.0),
            np.where(n == vocab - 1, 5.0, 0.0), -np.inf * np.ones(vocab), np.where(n < 3, 1.0, -np.inf),
            np.where(n % 2048 == 5, 4.0, np.sin(n))]
    for pad, offset in ((0, 0), (3, 1)):
        s = Mat(torch, len(rows), vocab, dtype, np.stack(rows), pad, offset)
        token = np.arange(len(rows)) * 7 % vocab
        for k in (1, 2, 13, 32):
            _forward(torch, v, s, token, k, dtype)


def test_logprob_gradient_against_differences(torch, v):  # noqa: F811
    rows, vocab, T, h = 6, 300, 0.8, 1e-2
    s, token, dev = _inputs(torch, rows, vocab, "float32", padding=0.3)
    g = _rng(8)
    d, dl, dh = (torch.as_tensor(g.standard_normal(n)).float().cuda() for n in ((rows, vocab), rows, rows))
    lp, ent, st, out = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda"), torch.empty_like(d)

    def f(x):
        v.vrcclLogProbForward(x.contiguous(), dev, lp, ent, st, None, None, rows, vocab, 0, "float32", "int64", T)
        return (dl.double() * lp.double() + dh.double() * ent.double()).sum().item()

    x = s.view.clone()
    f(x)
    v.vrcclLogProbBackward(x, dev, st, ent, dl, dh, out, rows, vocab, "float32", "int64", T)
    slope = (f(x + h * d) - f(x - h * d)) / (2 * h)
    # third differences of log sum exp and the entropy: a few |d / T|^3 each row, times h^2 / 6; rounding of some 40 EPS a value over h
    tol = rows * 30 * (1 / T) ** 3 * h * h / 6 * 4 + rows * 40 * EPS * 8 / h
    assert abs((out.double() * d.double()).sum().item() - slope) <= tol


def test_logprob_gradient_strides(torch, v):  # noqa: F811
    """One value of dlogprob and dentropy for all rows, and one every third."""
    rows, vocab = 7, 1003
    s, token, dev = _inputs(torch, rows, vocab, "bfloat16")
    _, entropy, stats = _forward(torch, v, s, token, 0, "bfloat16")
    wide = torch.randn(rows, 3, device="cuda")
    want, got = torch.empty(rows, vocab, device="cuda", dtype=torch.bfloat16), torch.empty(rows, vocab, device="cuda", dtype=torch.bfloat16)
    args = (rows, vocab, "bfloat16", "int64")
    v.vrcclLogProbBackward(s.ptr, dev, stats, entropy, wide[:, 0].contiguous(), wide[:, 1].contiguous(), want, *args)
    v.vrcclLogProbBackward(s.ptr, dev, stats, entropy, wide.data_ptr(), wide.data_ptr() + 4, got, *args, dlogprob_stride=3, dentropy_stride=3)
    assert torch.equal(want, got)
    v.vrcclLogProbBackward(s.ptr, dev, stats, entropy, torch.full((rows,), 0.5, device="cuda"), torch.full((rows,), 0.25, device="cuda"), want, *args)
    v.vrcclLogProbBackward(s.ptr, dev, stats, entropy, torch.full((1,), 0.5, device="cuda"), torch.full((1,), 0.25, device="cuda"), got, *args,
                           dlogprob_stride=0, dentropy_stride=0)
    assert torch.equal(want, got)


def test_logprob_same_bits_every_time(torch, v):  # noqa: F811
    """Split over clusters and not, in a graph, on another stream."""
    for rows, vocab in ((2, 131072), (300, 9000)):
        s, token, dev = _inputs(torch, rows, vocab, "bfloat16")
        outs = [torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda"),
                torch.empty(rows, 20, device="cuda"), torch.empty(rows, 20, device="cuda", dtype=torch.int32),
                torch.empty(rows, vocab, device="cuda", dtype=torch.bfloat16)]
        one = torch.ones(rows, device="cuda")

        def step(stream=None):
            v.vrcclLogProbForward(s.ptr, dev, *outs[:5], rows, vocab, 20, "bfloat16", "int64", stream=stream)
            v.vrcclLogProbBackward(s.ptr, dev, outs[2], outs[1], one, one, outs[5], rows, vocab, "bfloat16", "int64", stream=stream)

        step()
        want = [t.clone() for t in outs]
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for run in [graph.replay, lambda: step(side)] + 20 * [step]:
            for t in outs:
                t.zero_()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_logprob_of_no_vocabulary(torch, v):  # noqa: F811
    outs = [torch.full((3,), 7.0, device="cuda"), torch.full((3,), 7.0, device="cuda"), torch.full((3, 2), 7.0, device="cuda"),
            torch.full((3, 2), 7.0, device="cuda"), torch.full((3, 2), 7, device="cuda", dtype=torch.int32)]
    v.vrcclLogProbForward(None, torch.zeros(3, device="cuda", dtype=torch.int64), *outs, 3, 0, 2, "float32", "int64")
    assert all((t == 0).all() for t in outs[:3]) and (outs[3] == -float("inf")).all() and (outs[4] == -1).all()


def test_logprob_rows_beyond_32_bits(torch, v):  # noqa: F811
    ld, vocab = (1 << 31) + 8, 5000
    buf = torch.empty(2 * ld + vocab, device="cuda", dtype=torch.bfloat16)
    x = buf.as_strided((3, vocab), (ld, 1))
    x.copy_(torch.as_tensor(_rng(9).standard_normal((3, vocab))))
    flat, dev = x.clone(), torch.tensor([1, 4999, 2500], device="cuda")
    one = torch.ones(3, device="cuda")
    res = []
    for t in (x, flat):
        outs = [torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, 2, device="cuda"),
                torch.empty(3, 5, device="cuda"), torch.empty(3, 5, device="cuda", dtype=torch.int32)]
        v.vrcclLogProbForward(t, dev, *outs, 3, vocab, 5, "bfloat16", "int64")
        v.vrcclLogProbBackward(t, dev, outs[2], outs[1], one, one, t, 3, vocab, "bfloat16", "int64")
        res.append(outs + [t.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("vocab,pad,offset", [(40, 0, 0), (257, 1, 0), (1003, 0, 3), (1891, 8, 1), (2048, 0, 0), (4090, 3, 0)])
def test_logprob_of_many_short_rows(torch, v, vocab, pad, offset, dtype):  # noqa: F811
    """A warp a row: masks, ties (too many to collect, too), padding, every length of the list."""
    E = 4 if dtype == "float32" else 2
    rows = max(80, vocab * E // 8 + 5)
    s, token, _ = _inputs(torch, rows, vocab, dtype, pad, offset)
    low, a = float(torch.finfo(getattr(torch, dtype)).min), s.view
    a[1] = 1.5
    a[2] = (a[2] * 0.5).round()
    a[3, ::2] = -float("inf")
    a[4] = -float("inf")
    a[5] = low
    a[6, 1:] = -float("inf")
    a[7, : vocab // 2] = 0.0
    a[7, vocab // 3: vocab // 2] = -0.0
    a[7, vocab // 2:] = -1.0
    a[8] = -3.0
    a[8, vocab - 1] = a[8, 0] = a[8, vocab // 2] = 2.0
    a[9, : vocab - 5] = -float("inf")
    token[[1, 4, 8]] = 0, vocab - 1, vocab // 2
    for k, T in ((1, 1.0), (5, 0.7), (32, 2.0), (0, 1.0), (17, 1.0)):
        _forward(torch, v, s, token, k, dtype, T)


@pytest.mark.parametrize("dtype,vocab", [("bfloat16", 2419), ("float16", 4000), ("float32", 3585), ("bfloat16", 8191)])
def test_lists_as_long_as_a_row_has_segments(torch, v, dtype, vocab):  # noqa: F811
    """Around the number of a row's 512-byte pieces, which are counted in fours."""
    s, token, _ = _inputs(torch, 15, vocab, dtype, padding=0.1)
    for k in range(vocab * (4 if dtype == "float32" else 2) // 512 - 2, vocab * (4 if dtype == "float32" else 2) // 512 + 5):
        if 0 < k <= 32:
            _forward(torch, v, s, token, k, dtype)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("vocab,pad,opad,oskew", [(5, 0, 0, 0), (257, 1, 1, 0), (1003, 0, 3, 3), (1347, 3, 3, 0), (2048, 0, 8, 0)])
def test_logprob_gradient_of_many_short_rows(torch, v, vocab, pad, opad, oskew, dtype):  # noqa: F811
    s, token, _ = _inputs(torch, 1300, vocab, dtype, pad)
    s.view[7] = -float("inf")
    s.view[8, ::2] = -float("inf")
    token[8] = vocab - 1 if vocab % 2 == 0 else 1
    dev, entropy, stats = _forward(torch, v, s, token, 0, dtype, 0.9)
    _backward(torch, v, s, token, dev, entropy, stats, dtype, 0.9, opad, oskew)
    _backward(torch, v, s, token, dev, entropy, stats, dtype, 0.9, in_place=True)


def test_short_rows_that_are_not_finite(torch, v):  # noqa: F811
    """Rows of a NaN or infinity among many give what they give among few, which go another way."""
    rows, vocab, k = 600, 1001, 6
    x = torch.as_tensor(_rng(8).standard_normal((rows, vocab))).float().cuda()
    x[1, 77] = x[2, 5] = x[2, 999] = float("inf")
    x[3, 9] = float("inf")
    x[3, 300] = x[3, 200] = x[4, 1000] = x[0, 0] = float("nan")
    token = torch.arange(rows, device="cuda")

    def call(n):
        f = [torch.empty(n, device="cuda") for _ in range(2)]
        stats, top, index = torch.empty(n, 2, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, k, device="cuda", dtype=torch.int32)
        v.vrcclLogProbForward(x[:n], token[:n], f[0], f[1], stats, top, index, n, vocab, k, "float32", "int64")
        return f, top, index

    (few, ft, fi), (many, mt, mi) = call(5), call(rows)
    assert torch.equal(mi[:5], fi)
    for p, q in zip([*many, mt], [*few, ft]):
        assert torch.isnan(p[:5]).equal(torch.isnan(q)) and torch.isfinite(p[5:]).all()
    assert torch.isnan(many[0][:5]).all() and fi[4, 0] == 1000 and fi[3, :3].tolist() == [200, 300, 9] and fi[2, :2].tolist() == [5, 999]
