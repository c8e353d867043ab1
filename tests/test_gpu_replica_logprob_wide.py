"""Token log probabilities of wide vocabularies on the GPU, and of rows that go
a warp each beside the same rows that go a block each: values against 64 bits,
the alternatives' order against keys that are sorted as integers, both computed
by torch on the GPU, so that rows may be long. Tolerances as in
test_gpu_replica_logprob.py, of whole matrices."""
import pytest

from test_gpu_replica_ops import EPS, FLOATS, torch, v  # noqa: F401

pytestmark = pytest.mark.gpu


def _order(torch, x, k):  # noqa: F811
    """Indices of the k largest entries, equal ones by the lowest index, a NaN above everything."""
    x = x.float() + 0.0  # (zeros alike)
    bits = x.view(torch.int32).long() & 0xFFFFFFFF
    bits = torch.where(torch.isnan(x), torch.full_like(bits, 0x7FFFFFFF), bits)
    value = torch.where(bits >> 31 > 0, ~bits & 0xFFFFFFFF, bits | 0x80000000)
    key = value << 31 | (1 << 31) - 1 - torch.arange(x.shape[1], device="cuda")
    return ((1 << 31) - 1 - (key.topk(k, 1)[0] & (1 << 31) - 1)).int()


def _check(torch, v, x, token, k, T=1.0):  # noqa: F811
    rows, vocab = x.shape
    f = [torch.full((rows,), 7.0, device="cuda") for _ in range(2)]
    stats, top = torch.full((rows, 2), 7.0, device="cuda"), torch.full((rows, k), 7.0, device="cuda")
    index = torch.full((rows, k), 7, device="cuda", dtype=torch.int32)
    v.vrcclLogProbForward(x, token, *f, stats, top, index, rows, vocab, k, x.dtype, "int64", T)
    for at in range(0, rows, 64):
        r = slice(at, at + 64)
        given = (token[r] >= 0) & (token[r] < vocab)
        want = torch.where(given[:, None], _order(torch, x[r], k), -1)
        assert torch.equal(index[r], want), f"rows {at}..: {(index[r] != want).any(1).nonzero().flatten().tolist()}"
        s = x[r].double()
        most = s.amax(1, keepdim=True)
        z = (s - most) / T
        e = z.exp()
        total = e.sum(1)
        seen = torch.where(e > 0, z.abs(), 0.0)
        known = torch.where(e > 0, z, 0.0)
        n = vocab / 32 + 64  # (a warp a row: a lane's share, and the joins)
        el = (n + ((3 * seen + 4) * e).sum(1) / total) * EPS
        ew = (((n + 8 + 3 * seen) * seen * e).sum(1) / total) * EPS + el * (seen * e).sum(1) / total
        ll = total.log()
        tl, te = el + 2 * EPS * ll.abs(), ew + el + 4 * EPS * ll.abs()
        entropy = ll - (e * known).sum(1) / total
        fine = given & torch.isfinite(most[:, 0]) & torch.isfinite(total)
        q = z - ll[:, None]
        lp, best = q.gather(1, token[r].clamp(0, vocab - 1)[:, None])[:, 0], q.gather(1, index[r].clamp(min=0).long())
        far = lambda w: 4 * EPS * (w.abs() + ll.abs().reshape(-1, *[1] * (w.ndim - 1)))  # noqa: E731

        def close(got, want, tol, what):
            want = torch.where(want < -float(torch.finfo(torch.float32).max), -float("inf"), want)  # (beyond binary32)
            equal = got.double() == want
            assert (equal | ((got - want).abs() <= tol))[fine].all(), what

        close(f[1][r], entropy, te, "entropy")
        close(stats[r, 0], most[:, 0], 0 * tl, "largest")
        close(stats[r, 1], ll, tl, "log sum")
        close(f[0][r], lp, tl + far(lp), "logprob")
        close(top[r], best, tl[:, None] + far(best), "alternatives")
        assert all((t[r][~given] == 0).all() for t in (*f, stats)) and (top[r][~given] == -float("inf")).all()
        nan = given & (torch.isnan(s).any(1) | (most[:, 0] == float("inf")))
        assert torch.isnan(f[0][r][nan]).all() and torch.isnan(f[1][r][nan]).all()
        none = given & (most[:, 0] == -float("inf"))
        assert (f[0][r][none] == -float("inf")).all() and (f[1][r][none] == 0).all() and (top[r][none] == -float("inf")).all()
    return index


def _rows(torch, rows, vocab, dtype, seed=1):  # noqa: F811
    """Rows of noise, the first of them with ties, masks and maxima where segments begin and end."""
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, vocab, generator=gen, device="cuda").mul_(2.5).to(getattr(torch, dtype))
    token = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    inf, n = float("inf"), torch.arange(vocab, device="cuda")
    special = [lambda a: a.mul_(0.5).round_(),                                   # few values
               lambda a: a.fill_(1.5),                                           # one
               lambda a: a[: vocab - 9].fill_(-inf),                             # the last few
               lambda a: a[vocab // 3: 2 * vocab // 3].fill_(-inf),              # a hole
               lambda a: a[vocab - 40:].add_(30.0),                              # all in the last segment, which is not whole
               lambda a: a[:40].add_(30.0),
               lambda a: a[::2].fill_(-inf),
               lambda a: a.copy_((n % 4096 < 3).to(a.dtype)),                    # ties, one segment in some
               lambda a: a.copy_(torch.where(n % 1024 == 1023, 4.0, -1.0)),
               lambda a: a.fill_(-inf),
               lambda a: a.copy_((n.clamp(max=2000) / 16)),
               lambda a: a.copy_(-(n.clamp(max=2000) / 16)),
               lambda a: a[1:].fill_(torch.finfo(a.dtype).min),
               lambda a: a.index_fill_(0, torch.tensor([5, vocab // 2, vocab - 1], device="cuda"), inf),
               lambda a: a.index_fill_(0, torch.tensor([7, vocab // 2 + 1, vocab - 2], device="cuda"), float("nan")),
               lambda a: a[vocab // 2: vocab // 2 + 600].add_(20.0)]             # all in one segment, or two
    for a, change in zip(x, special):
        change(a)
    token[9], token[-1] = 0, -1
    return x, token


@pytest.mark.parametrize("dtype,vocab", [("bfloat16", 131072), ("float16", 140001), ("float32", 131072), ("float32", 70001), ("float32", 300001),
                                         ("bfloat16", 600007)])
def test_alternatives_of_rows_a_block_each(torch, v, dtype, vocab):  # noqa: F811
    """More rows than blocks are split for: segments of two, four and eight loads."""
    x, token = _rows(torch, 330, vocab, dtype)
    for k, T in ((1, 1.0), (8, 0.7), (32, 1.0)):
        _check(torch, v, x, token, k, T)


@pytest.mark.parametrize("rows,vocab,dtype", [(17, 1100001, "float32"), (17, 4200003, "float32"), (16, 8000001, "bfloat16"), (120, 600007, "bfloat16")])
def test_alternatives_of_split_rows_of_long_segments(torch, v, rows, vocab, dtype):  # noqa: F811
    """Rows over clusters, whose blocks have segments of two loads to sixteen."""
    x, token = _rows(torch, rows, vocab, dtype, 2)
    for k in (8, 32):
        _check(torch, v, x, token, k)


@pytest.mark.parametrize("dtype,vocab", [("bfloat16", 131072), ("float32", 300001)])
def test_alternatives_do_not_depend_on_how_rows_are_split(torch, v, dtype, vocab):  # noqa: F811
    x, token = _rows(torch, 330, vocab, dtype, 3)
    many = _check(torch, v, x, token, 20)
    for n in (1, 17, 100, 200):
        assert torch.equal(_check(torch, v, x[:n], token[:n].clamp(min=0), 20), many[:n])


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("vocab", [2100, 4093])
def test_rows_a_warp_each_and_a_block_each(torch, v, vocab, dtype):  # noqa: F811
    """Rows of 4 to 16 KB: enough of them go a warp each, a few a block each; infinities and NaN among them."""
    if dtype != "float32":
        vocab *= 2
    x, token = _rows(torch, vocab // 2 + 9, vocab, dtype, 4)
    for k in (1, 6, 32):
        many = _check(torch, v, x, token, k)
        for n in (5, 17):
            assert torch.equal(_check(torch, v, x[:n], token[:n].clamp(min=0), k), many[:n])
