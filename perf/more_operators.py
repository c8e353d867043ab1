"""More operators of a data-parallel replica, as they are measured: dropout
from a counter-based generator with the residual's addition, RMS norm with the
residual's addition and an 8-bit output, and log probabilities of given tokens
with entropy and top alternatives, each forward and backward.

A case names an operator (``op``), a direction (``dir``) and the sizes; rows
are tokens. ``pad`` is how many elements a row's stride exceeds its length
by, so an odd pad gives rows that start on no vector boundary.
"""
import math

import torch

own = False

EPS = 1e-5
DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
SIZE = {"bfloat16": 2, "float16": 2, "float32": 4}
LARGEST = {"int8": 127.0, "e4m3": 448.0}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases

def _dropout(dir, rows, cols, dtype, p, residual=False, pad=0):
    return {"op": "dropout", "dir": dir, "rows": rows, "cols": cols, "dtype": dtype, "p": p, "residual": residual,
            "pad": pad}


def _rms(dir, rows, cols, dtype, params, residual=True, quant="none", group=0, pad=0):
    """``residual``: forward adds it (and keeps the sum); backward adds the sum's own gradient."""
    return {"op": "rms", "dir": dir, "rows": rows, "cols": cols, "dtype": dtype, "params": params, "residual": residual,
            "quant": quant, "group": group, "pad": pad}


def _logprob(dir, rows, vocab, k, dtype, temperature=1.0, index="int64", empty=0.0, pad=0):
    return {"op": "logprob", "dir": dir, "rows": rows, "vocab": vocab, "k": k, "dtype": dtype, "temperature": temperature,
            "index": index, "empty": empty, "pad": pad}


def listed():
    def named(name, case):
        return dict(case, name=name)
    return [
        # a short piece of a sequence, one layer's branch added to the residual stream: latency
        named("dropout_fwd_few", _dropout("fwd", 64, 4096, "bfloat16", 0.1, residual=True)),
        # a micro-batch of 32k tokens, the branch dropped out and added
        named("dropout_fwd_large", _dropout("fwd", 32768, 4096, "bfloat16", 0.1, residual=True)),
        # the gradient in a view of a wider buffer: odd width, rows on no vector boundary
        named("dropout_bwd_odd", _dropout("bwd", 5003, 1001, "float16", 0.25, pad=6)),
        # a few tokens of a sequence being continued: latency
        named("rms_fwd_few", _rms("fwd", 4, 4096, "bfloat16", "bfloat16")),
        # a micro-batch's residual addition and norm, parameters held in fp32
        named("rms_fwd_large", _rms("fwd", 32768, 4096, "bfloat16", "float32")),
        # the same with the normed activations in 8 bits, a scale for each 128 columns
        named("rms_fwd_codes", _rms("fwd", 16384, 5120, "bfloat16", "bfloat16", quant="e4m3", group=128)),
        # odd sizes in fp32, rows on no vector boundary
        named("rms_bwd_odd", _rms("bwd", 3001, 2003, "float32", "float32", pad=3)),
        # a wide model's micro-batch, the residual stream's gradient added, fp32 parameters
        named("rms_bwd_large", _rms("bwd", 16384, 8192, "bfloat16", "float32")),
        # one step of four sequences being continued, with the alternatives that a server reports: latency
        named("logprob_fwd_few", _logprob("fwd", 4, 131072, 20, "bfloat16")),
        # a micro-batch scored over a large vocabulary
        named("logprob_fwd_large", _logprob("fwd", 4096, 131072, 8, "bfloat16")),
        # odd vocabulary in fp32 at a sampling temperature, a fifth of the positions padding
        named("logprob_fwd_odd", _logprob("fwd", 1021, 50001, 5, "float32", 0.7, index="int32", empty=0.2)),
        # the gradient of a policy's loss with an entropy term
        named("logprob_bwd_large", _logprob("bwd", 4096, 131072, 0, "bfloat16")),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths are a power of two times 1, 5/4 or 7/4, as most models' are; the others are odd."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.5:
        return min(hi, max(lo, (1 << n.bit_length() - 3) * rng.choice([4, 5, 7])))
    return n | 1


def draw(rng):
    op = rng.choice(["dropout", "rms", "logprob"])
    dir = rng.choice(["fwd", "bwd"])
    dtype = rng.choice(["bfloat16", "float16", "float32"])
    pad = rng.choice([0, 0, 8, 3])
    rows = _log(rng, 1, 32768)
    if op == "logprob":
        vocab = _width(rng, 1000, 131072)
        return _logprob(dir, max(1, min(rows, (1 << 28) // vocab)), vocab, rng.choice([0, 1, _log(rng, 2, 32)]), dtype,
                        rng.choice([0.7, 1.0, 2.0]), rng.choice(["int32", "int64"]), rng.choice([0.0, 0.1]), pad)
    cols = _width(rng, 64, 16384)
    rows = min(rows, (1 << 26) // cols)
    if op == "dropout":
        return _dropout(dir, rows, cols, dtype, rng.choice([0.05, 0.1, 0.25, 0.5]), rng.random() < 0.5 and dir == "fwd", pad)
    quant = rng.choice(["none", "none", "int8", "e4m3"]) if dir == "fwd" else "none"
    return _rms(dir, rows, cols, dtype, rng.choice([dtype, "float32"]), rng.random() < 0.5, quant,
                0 if quant == "none" else rng.choice([0, 32, 64, 128]), pad)


# ------------------------------------------------------------------ inputs

def _rows(gen, rows, cols, pad, dtype, scale=1.0):
    t = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=DT[dtype])
    if scale != 1.0:
        t.mul_(scale)
    return t[:, :cols]


def _empty(rows, cols, pad, dtype):
    return torch.empty(rows, cols + pad, device="cuda", dtype=dtype)[:, :cols]


def _groups(case):
    return 1 if not case["group"] else -(-case["cols"] // case["group"])


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    c, dt, pad = case, case["dtype"], case["pad"]
    f32 = {"device": "cuda", "dtype": torch.float32}
    if c["op"] == "dropout":
        n, w = c["rows"], c["cols"]
        s["x"] = _rows(gen, n, w, pad, dt)
        s["r"] = _rows(gen, n, w, pad, dt, 1.5) if c["residual"] else None
        s["y"] = _empty(n, w, pad, DT[dt])
        # the step's seed lives on the GPU, a captured graph reads it anew; the offset tells a step's layers apart
        s["seed"] = torch.randint(-(1 << 62), 1 << 62, (1,), generator=gen, device="cuda")
        s["offset"], s["first_row"] = 7 + (seed % 1000), 4096 * (seed % 3)
    elif c["op"] == "rms":
        n, w = c["rows"], c["cols"]
        s["gamma"] = (1 + 0.1 * torch.randn(w, generator=gen, **f32)).to(DT[c["params"]])
        s["x"] = _rows(gen, n, w, pad, dt)
        if c["dir"] == "fwd":
            s["r"] = _rows(gen, n, w, pad, dt, 1.5) if c["residual"] else None
            s["sum"] = _empty(n, w, pad, DT[dt]) if c["residual"] else None
            s["rstd"] = torch.empty(n, **f32)
            if c["quant"] == "none":
                s["y"] = _empty(n, w, pad, DT[dt])
            else:
                s["codes"], s["scales"] = _empty(n, w, pad, CODES[c["quant"]]), torch.empty(n, _groups(c), **f32)
        else:
            s["dy"] = _rows(gen, n, w, pad, dt)
            s["dsum"] = _rows(gen, n, w, pad, dt) if c["residual"] else None
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dx"], s["dgamma"] = _empty(n, w, pad, DT[dt]), torch.empty_like(s["gamma"])
    else:
        n, v, k = c["rows"], c["vocab"], c["k"]
        s["logits"] = _rows(gen, n, v, pad, dt, 2.5)
        token = (torch.rand(n, generator=gen, **f32) * v).long().clamp_(0, v - 1)
        if c["empty"]:
            token[torch.rand(n, generator=gen, **f32) < c["empty"]] = -100  # padding
        s["token"] = token.to(torch.int32) if c["index"] == "int32" else token
        if c["dir"] == "fwd":
            s["logprob"], s["entropy"], s["stats"] = torch.empty(n, **f32), torch.empty(n, **f32), torch.empty(n, 2, **f32)
            s["top"], s["top_index"] = torch.empty(n, k, **f32), torch.empty(n, k, device="cuda", dtype=torch.int32)
        else:
            s["dlogprob"] = torch.randn(n, generator=gen, **f32) / n
            s["dentropy"] = 0.01 * torch.rand(n, generator=gen, **f32) / n
            s["stats"], s["entropy"] = _stats(s)
            s["dlogits"] = _empty(n, v, pad, DT[dt])
    return s


# ------------------------------------------------------------------ plain forms

def _philox(seed, offset, groups):
    """The 128 bits of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; 2011) under
    the key ``seed`` for the counters (group, offset), as four tensors of 32 bits each in int64."""
    low = 0xFFFFFFFF
    k0, k1 = seed & low, seed >> 32 & low
    a, b = groups & low, groups >> 32 & low
    c, d = torch.full_like(a, offset & low), torch.full_like(a, offset >> 32 & low)
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32 & low) ^ b ^ k0, q & low, (p >> 32 & low) ^ d ^ k1, p & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return a, b, c, d


def _mask(s):
    """(kept, what a kept element is multiplied by): 16 bits decide an element."""
    per = -(-s["cols"] // 8)
    rows = s["first_row"] + torch.arange(s["rows"], device="cuda")
    words = torch.stack(_philox(s["seed"], s["offset"], rows[:, None] * per + torch.arange(per, device="cuda")), 2)
    bits = torch.stack([words & 0xFFFF, words >> 16], 3).view(s["rows"], per * 8)[:, :s["cols"]]
    drop = math.floor(s["p"] * 65536 + 0.5)
    return bits >= drop, 65536 / (65536 - drop)


def _plain_dropout(s):
    kept, scale = _mask(s)
    y = torch.where(kept, s["x"].float() * scale, 0.0)
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(DT[s["dtype"]])


def _plain_rms_fwd(s):
    dt = DT[s["dtype"]]
    x = s["x"].float()
    if s["r"] is not None:
        x = (x + s["r"].float()).to(dt).float()
    rstd = torch.rsqrt(x.square().mean(1) + EPS)
    y = x * rstd[:, None] * s["gamma"].float()
    out = {"rstd": rstd} if s["r"] is None else {"rstd": rstd, "sum": x.to(dt)}
    if s["quant"] == "none":
        return dict(out, y=y.to(dt))
    group = s["group"] or s["cols"]
    wide = torch.nn.functional.pad(y, (0, _groups(s) * group - s["cols"])).view(s["rows"], -1, group)
    scales = wide.abs().amax(2) / LARGEST[s["quant"]]
    codes = wide / scales[:, :, None]
    codes = codes.round().clamp(-127, 127) if s["quant"] == "int8" else codes.to(torch.float8_e4m3fn).float()
    return dict(out, scales=scales, values=_values(codes, scales, s))


def _values(codes, scales, s):
    """The values that codes [rows, groups, columns] stand for."""
    return (codes * scales[:, :, None]).to(torch.bfloat16).view(s["rows"], -1)[:, :s["cols"]]


def _plain_rms_bwd(s):
    rstd = s["rstd"][:, None]
    xh, dy = s["x"].float() * rstd, s["dy"].float()
    g = dy * s["gamma"].float()
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(DT[s["dtype"]]), "dgamma": (dy * xh).sum(0).to(DT[s["params"]])}


def _given(s):
    return (s["token"] >= 0) & (s["token"] < s["vocab"])


def _stats(s):
    """((largest logit, log of the sum of exp((logit - largest) / temperature)), entropy) of each row; 0 for padding."""
    x = s["logits"].float()
    top = x.amax(1)
    x = (x - top[:, None]) / s["temperature"]
    e = torch.exp(x)
    total = e.sum(1)
    entropy = total.log() - (e * x).sum(1) / total
    return torch.where(_given(s)[:, None], torch.stack([top, total.log()], 1), 0.0), torch.where(_given(s), entropy, 0.0)


def _plain_logprob_fwd(s):
    given, k = _given(s), min(s["k"], s["vocab"])
    stats, entropy = _stats(s)
    log = lambda x: (x.float() - stats[:, :1]) / s["temperature"] - stats[:, 1:]  # noqa: E731
    token = torch.where(given, s["token"].long(), 0)[:, None]
    out = {"logprob": torch.where(given, log(s["logits"].gather(1, token))[:, 0], 0.0), "entropy": entropy, "stats": stats}
    if k:
        x, at = s["logits"].sort(dim=1, descending=True, stable=True)
        out["top"] = torch.where(given[:, None], log(x[:, :k]), -math.inf)
        out["top_index"] = torch.where(given[:, None], at[:, :k], -1).to(torch.int32)
    return out


def _plain_logprob_bwd(s):
    logq = (s["logits"].float() - s["stats"][:, :1]) / s["temperature"] - s["stats"][:, 1:]
    given = _given(s)
    dl, dh = (torch.where(given, s[name], 0.0)[:, None] / s["temperature"] for name in ("dlogprob", "dentropy"))
    d = torch.exp(logq) * -(dl + dh * (logq + s["entropy"][:, None]))
    d = d.scatter_add(1, torch.where(given, s["token"].long(), 0)[:, None], dl)
    return d.to(DT[s["dtype"]])


_PLAIN = {("dropout", "fwd"): _plain_dropout, ("dropout", "bwd"): _plain_dropout, ("rms", "fwd"): _plain_rms_fwd,
          ("rms", "bwd"): _plain_rms_bwd, ("logprob", "fwd"): _plain_logprob_fwd, ("logprob", "bwd"): _plain_logprob_bwd}


# ------------------------------------------------------------------ the framework's calls

def _own_dropout_fwd(s, v):
    v.vrcclDropoutForward(s["x"], s["r"], s["y"], s["rows"], s["cols"], s["dtype"], s["p"], s["seed"], s["offset"],
                          s["first_row"])
    return s["y"]


def _own_dropout_bwd(s, v):
    v.vrcclDropoutBackward(s["x"], s["y"], s["rows"], s["cols"], s["dtype"], s["p"], s["seed"], s["offset"], s["first_row"])
    return s["y"]


def _own_rms_fwd(s, v):
    out = {"rstd": s["rstd"]} if s["r"] is None else {"rstd": s["rstd"], "sum": s["sum"]}
    if s["quant"] == "none":
        v.vrcclRmsNormForward(s["x"], s["r"], s["gamma"], s["sum"], s["y"], s["rstd"], s["rows"], s["cols"], s["dtype"],
                              s["params"], EPS)
        return dict(out, y=s["y"])
    v.vrcclRmsNormForward(s["x"], s["r"], s["gamma"], s["sum"], None, s["rstd"], s["rows"], s["cols"], s["dtype"], s["params"],
                          EPS, s["codes"], s["scales"], s["quant"], s["group"])
    # what the codes stand for: a product of the reader's
    group = s["group"] or s["cols"]
    codes = s["codes"] if s["quant"] == "int8" else s["codes"].bfloat16()
    if s["cols"] % group:
        codes = torch.nn.functional.pad(codes, (0, _groups(s) * group - s["cols"]))
    return dict(out, scales=s["scales"], values=_values(codes.unflatten(1, (-1, group)), s["scales"], s))


def _own_rms_bwd(s, v):
    if "scratch" not in s:  # kept with the buffers from the first call on
        s["scratch"] = torch.empty(max(16, v.vrcclRmsNormWorkspace(s["rows"], s["cols"])), device="cuda", dtype=torch.uint8)
    v.vrcclRmsNormBackward(s["dy"], s["dsum"], s["x"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["rows"], s["cols"],
                           s["dtype"], s["params"], s["scratch"], s["scratch"].numel())
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def _own_logprob_fwd(s, v):
    top, at = (s["top"], s["top_index"]) if s["k"] else (None, None)
    v.vrcclLogProbForward(s["logits"], s["token"], s["logprob"], s["entropy"], s["stats"], top, at, s["rows"], s["vocab"],
                          s["k"], s["dtype"], s["token"].dtype, s["temperature"])
    out = {"logprob": s["logprob"], "entropy": s["entropy"], "stats": s["stats"]}
    return dict(out, top=top, top_index=at) if s["k"] else out


def _own_logprob_bwd(s, v):
    v.vrcclLogProbBackward(s["logits"], s["token"], s["stats"], s["entropy"], s["dlogprob"], s["dentropy"], s["dlogits"],
                           s["rows"], s["vocab"], s["dtype"], s["token"].dtype, s["temperature"])
    return s["dlogits"]


_OWN = {("dropout", "fwd"): _own_dropout_fwd, ("dropout", "bwd"): _own_dropout_bwd, ("rms", "fwd"): _own_rms_fwd,
        ("rms", "bwd"): _own_rms_bwd, ("logprob", "fwd"): _own_logprob_fwd, ("logprob", "bwd"): _own_logprob_bwd}


def run(s):
    if own:
        from ring_allreduce_reduction_gb300 import vrccl
        return _OWN[s["op"], s["dir"]](s, vrccl)
    return _PLAIN[s["op"], s["dir"]](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        return {"bytes": (2 + c["residual"]) * n * e, "flops": 8 * n}  # the generator's steps, an eighth of 64 an element
    if c["op"] == "rms":
        n, params = c["rows"] * c["cols"], c["cols"] * SIZE[c["params"]]
        if c["dir"] == "bwd":
            return {"bytes": (3 + c["residual"]) * n * e + 4 * c["rows"] + 2 * params, "flops": 10 * n}
        out = n * e if c["quant"] == "none" else n + 4 * c["rows"] * _groups(c)
        return {"bytes": n * e * (3 if c["residual"] else 1) + out + 4 * c["rows"] + params, "flops": 5 * n}
    n, v, k = c["rows"], c["vocab"], c["k"]
    ids = n * (4 if c["index"] == "int32" else 8)
    given = n * (1 - c["empty"])  # padding needs no logits read
    if c["dir"] == "fwd":
        return {"bytes": int(given * v * e) + ids + n * (16 + 8 * k), "flops": 6 * n * v}
    return {"bytes": int((given + n) * v * e) + ids + n * 20, "flops": 7 * n * v}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_dropout(s):
    # the generator once more, its 32 x 32-bit products from 16-bit halves
    def product(x, m):
        lo, hi = x % 65536, x // 65536
        cross = lo * (m // 65536) + (lo * (m % 65536) // 65536) + (hi * (m % 65536)) % 65536
        high = hi * (m // 65536) + hi * (m % 65536) // 65536 + cross // 65536
        return high % 2 ** 32, cross % 65536 * 65536 + lo * (m % 65536) % 65536

    seed = int(s["seed"].item()) % 2 ** 64
    per = (s["cols"] + 7) // 8
    group = torch.arange(s["first_row"] * per, (s["first_row"] + s["rows"]) * per, device="cuda")
    c = [group % 2 ** 32, group // 2 ** 32, torch.full_like(group, s["offset"] % 2 ** 32), torch.full_like(group, s["offset"] // 2 ** 32)]
    for i in range(10):
        h0, l0 = product(c[0], 0xD2511F53)
        h1, l1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ (seed + i * 0x9E3779B9) % 2 ** 32, l1, h0 ^ c[3] ^ (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32, l0]
    u = torch.stack([c[j // 2] // 65536 if j % 2 else c[j // 2] % 65536 for j in range(8)], 1).view(s["rows"], per * 8)
    drop = math.floor(s["p"] * 65536 + 0.5)
    y = s["x"].double() * (u[:, :s["cols"]] >= drop) / (1 - drop / 65536)
    return y if s["r"] is None else y + s["r"].double()


def _exact_codes(y, quant, group):
    """(scales, values) by the definition: a step is 2^-3 of a value's power of two, at least 2^-9; or 1."""
    parts = [y[:, at:at + group] for at in range(0, y.shape[1], group)]
    scales = torch.stack([p.abs().amax(1) for p in parts], 1) / LARGEST[quant]
    values = []
    for p, scale in zip(parts, scales.t()):
        v = p / scale[:, None]
        step = 1.0 if quant == "int8" else torch.exp2(torch.frexp(v)[1].clamp(min=-5).double() - 4)
        values.append((v / step).round() * step * scale[:, None])
    return scales, torch.cat(values, 1)


def _exact_rms(s):
    x, gamma = s["x"].double(), s["gamma"].double()
    if s["dir"] == "fwd":
        if s["r"] is not None:
            x = (x + s["r"].double()).to(DT[s["dtype"]]).double()
        rstd = (x.pow(2).sum(1) / s["cols"] + EPS) ** -0.5
        y = x * rstd[:, None] * gamma
        out = {"rstd": rstd} if s["r"] is None else {"rstd": rstd, "sum": x}
        if s["quant"] == "none":
            return dict(out, y=y)
        scales, values = _exact_codes(y, s["quant"], s["group"] or s["cols"])
        return dict(out, scales=scales, values=values)
    gamma.requires_grad_()
    dx = []
    for at in range(0, s["rows"], 4096):
        part = x[at:at + 4096].requires_grad_()
        y = part / torch.sqrt(part.pow(2).sum(1, keepdim=True) / s["cols"] + EPS) * gamma
        y.backward(s["dy"][at:at + 4096].double())
        dx.append(part.grad)
    dx = torch.cat(dx)
    return {"dx": dx if s["dsum"] is None else dx + s["dsum"].double(), "dgamma": gamma.grad}


def _exact_logprob(s):
    T, k, out = s["temperature"], min(s["k"], s["vocab"]), []
    for at in range(0, s["rows"], 256):
        rows = slice(at, at + 256)
        logits, given = s["logits"][rows].double().requires_grad_(), _given(s)[rows]
        logq = torch.log_softmax(logits / T, 1)
        logprob = logq.gather(1, s["token"][rows].long().clamp(0, s["vocab"] - 1)[:, None])[:, 0]
        entropy = -(torch.exp(logq) * logq).sum(1)
        if s["dir"] == "bwd":
            loss = (torch.where(given, s["dlogprob"][rows].double() * logprob + s["dentropy"][rows].double() * entropy, 0.0)).sum()
            out.append([torch.autograd.grad(loss, logits)[0]])
            continue
        x = logits.detach()
        most = x.amax(1)
        stats = torch.stack([most, torch.logsumexp(x / T, 1) - most / T], 1)
        got = [torch.where(given, logprob, 0.0), torch.where(given, entropy, 0.0), torch.where(given[:, None], stats, 0.0)]
        if k:
            # the k-th largest logit, then the first k of those not below it in the order (value, lowest index)
            edge = x.topk(k, 1)[0][:, -1:]
            best = torch.where(x >= edge, x, -math.inf).topk(min(s["vocab"], k + 96), 1)[1].sort(1)[0]
            order = x.gather(1, best).sort(dim=1, descending=True, stable=True)[1][:, :k]
            index = best.gather(1, order)
            got += [torch.where(given[:, None], logq.gather(1, index), -math.inf), None]
        out.append([None if t is None else t.detach() for t in got])
    if s["dir"] == "bwd":
        return torch.cat([t[0] for t in out])
    names = ("logprob", "entropy", "stats", "top", "top_index")
    return {name: None if t[0] is None else torch.cat(t) for name, t in zip(names, zip(*out))}


def exact(case, seed):
    return {"dropout": _exact_dropout, "rms": _exact_rms, "logprob": _exact_logprob}[case["op"]](prepare(case, seed))
