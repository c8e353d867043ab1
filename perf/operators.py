"""The operators a data-parallel replica runs between two AllReduces, as they
are measured: layer norm, the linear layer with its epilogue, and the
distillation loss, each forward and backward.

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


# ------------------------------------------------------------------ cases

def _norm(dir, rows, cols, dtype, params, pad=0):
    return {"op": "norm", "dir": dir, "rows": rows, "cols": cols, "dtype": dtype, "params": params, "pad": pad}


def _linear(dir, rows, outs, ins, dtype, act, residual=False, pad=0):
    return {"op": "linear", "dir": dir, "rows": rows, "outs": outs, "ins": ins, "dtype": dtype, "act": act,
            "residual": residual, "pad": pad}


def _distill(dir, rows, vocab, k, dtype, temperature, index="int64", empty=0.0, pad=0):
    return {"op": "distill", "dir": dir, "rows": rows, "vocab": vocab, "k": k, "dtype": dtype,
            "temperature": temperature, "index": index, "empty": empty, "pad": pad}


def listed():
    def named(name, case):
        return dict(case, name=name)
    return [
        # a few tokens of a sequence being continued: latency
        named("norm_fwd_few", _norm("fwd", 4, 4096, "bfloat16", "bfloat16")),
        # a micro-batch of 32k tokens, parameters held in fp32
        named("norm_fwd_large", _norm("fwd", 32768, 4096, "bfloat16", "float32")),
        # a view of a wider activation: odd width, rows on no vector boundary
        named("norm_bwd_odd", _norm("bwd", 5003, 1001, "float16", "float16", pad=6)),
        # a wide model's micro-batch, gradients of the fp32 parameters
        named("norm_bwd_large", _norm("bwd", 16384, 8192, "bfloat16", "float32")),
        # one token: the weights are read once, nothing else counts
        named("linear_fwd_token", _linear("fwd", 1, 4096, 4096, "bfloat16", "gelu")),
        # the wide projection of a feed-forward block in training (keeps the pre-activation)
        named("linear_fwd_large", _linear("fwd", 8192, 8192, 2048, "bfloat16", "gelu_tanh")),
        # ragged sizes, no operand's rows aligned, a residual added in the epilogue
        named("linear_fwd_odd", _linear("fwd", 1021, 1003, 517, "float16", "silu", residual=True)),
        # both gradients of a square projection
        named("linear_bwd_large", _linear("bwd", 8192, 4096, 4096, "bfloat16", "gelu")),
        # a few positions scored over a large vocabulary: latency
        named("distill_fwd_few", _distill("fwd", 4, 131072, 64, "bfloat16", 2.0)),
        # a micro-batch's loss over a large vocabulary
        named("distill_fwd_large", _distill("fwd", 4096, 131072, 64, "bfloat16", 2.0)),
        # odd vocabulary in fp32, a fifth of the positions padding
        named("distill_bwd_odd", _distill("bwd", 301, 50001, 33, "float32", 1.0, index="int32", empty=0.2)),
        # the gradient of a micro-batch's loss
        named("distill_bwd_large", _distill("bwd", 4096, 131072, 128, "bfloat16", 2.0)),
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
    op = rng.choice(["norm", "linear", "distill"])
    dir = rng.choice(["fwd", "bwd"])
    dtype = rng.choice(["bfloat16", "float16", "float32"] if op != "linear" else ["bfloat16", "float16"])
    pad = rng.choice([0, 0, 8, 3])
    rows = _log(rng, 1, 8192)
    if op == "norm":
        cols = _width(rng, 64, 16384)
        rows = min(rows * 4, (1 << 26) // cols)
        return _norm(dir, rows, cols, dtype, rng.choice([dtype, "float32"]), pad)
    if op == "linear":
        outs, ins = _width(rng, 64, 8192), _width(rng, 64, 8192)
        rows = max(1, min(rows, (1 << 36) // (outs * ins)))
        return _linear(dir, rows, outs, ins, dtype, rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                       rng.random() < 0.5 and dir == "fwd", pad)
    vocab = _width(rng, 1000, 131072)
    return _distill(dir, max(1, min(rows, (1 << 28) // vocab)), vocab, _log(rng, 1, 256), dtype, rng.choice([1.0, 2.0, 4.0]),
                    rng.choice(["int32", "int64"]), rng.choice([0.0, 0.1]), pad)


# ------------------------------------------------------------------ inputs

def _rows(gen, rows, cols, pad, dtype, scale=1.0, shift=0.0):
    t = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=DT[dtype])
    if scale != 1.0:
        t.mul_(scale)
    if shift:
        t.add_(shift)
    return t[:, :cols]


def _empty(rows, cols, pad, dtype):
    return torch.empty(rows, cols + pad, device="cuda", dtype=DT[dtype])[:, :cols]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    c, dt, pad = case, case["dtype"], case["pad"]
    f32 = {"device": "cuda", "dtype": torch.float32}
    if c["op"] == "norm":
        n, w = c["rows"], c["cols"]
        s["x"] = _rows(gen, n, w, pad, dt, 1.5, 0.25)
        s["gamma"] = (1 + 0.1 * torch.randn(w, generator=gen, **f32)).to(DT[c["params"]])
        s["beta"] = (0.1 * torch.randn(w, generator=gen, **f32)).to(DT[c["params"]])
        if c["dir"] == "fwd":
            s["y"] = _empty(n, w, pad, dt)
            s["mean"], s["rstd"] = torch.empty(n, **f32), torch.empty(n, **f32)
        else:
            s["dy"] = _rows(gen, n, w, pad, dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
            s["dx"] = _empty(n, w, pad, dt)
            s["dgamma"], s["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])
    elif c["op"] == "linear":
        m, o, i = c["rows"], c["outs"], c["ins"]
        s["x"] = _rows(gen, m, i, pad, dt)
        s["w"] = _rows(gen, o, i, pad, dt, 1 / math.sqrt(i))
        if c["dir"] == "fwd":
            s["bias"] = (0.1 * torch.randn(o, generator=gen, **f32)).to(DT[dt])
            s["r"] = _rows(gen, m, o, pad, dt) if c["residual"] else None
            s["y"] = _empty(m, o, pad, dt)
            s["z"] = _empty(m, o, pad, dt) if c["act"] != "none" else None
        else:
            s["dy"] = _rows(gen, m, o, pad, dt)
            s["z"] = _rows(gen, m, o, pad, dt) if c["act"] != "none" else None
            s["dx"], s["dw"] = _empty(m, i, pad, dt), _empty(o, i, pad, dt)
            s["dbias"] = torch.empty(o, device="cuda", dtype=DT[dt])
    else:
        n, v, k = c["rows"], c["vocab"], c["k"]
        s["logits"] = _rows(gen, n, v, pad, dt, 2.5)
        # k distinct entries a row, the teacher's logits in falling order
        at = (torch.arange(k, device="cuda") + 0.999 * torch.rand(n, k, generator=gen, **f32)) * (v / k)
        at = at.long().clamp_(0, v - 1)
        s["teacher"] = (3 * torch.randn(n, k, generator=gen, **f32) + 8).sort(1, descending=True)[0].to(DT[dt])
        if c["empty"]:
            # padding positions have no entries; some others have fewer than k
            at[torch.rand(n, generator=gen, **f32) < c["empty"]] = -1
            at[torch.rand(n, k, generator=gen, **f32) < c["empty"] / 4] = -1
        s["index"] = at.to(torch.int32) if c["index"] == "int32" else at
        if c["dir"] == "fwd":
            s["loss"], s["stats"] = torch.empty(n, **f32), torch.empty(n, 2, **f32)
        else:
            s["dloss"] = torch.rand(n, generator=gen, **f32) / n
            s["stats"] = _distill_stats(s["logits"], s["index"], s["teacher"], c["temperature"])
            s["dlogits"] = _empty(n, v, pad, dt)
    return s


# ------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _kept(index, teacher, vocab):
    return (index >= 0) & (index < vocab) & (teacher > -math.inf)


def _distill_stats(logits, index, teacher, temperature):
    """(largest logit, log of the sum of exp((logit - largest) / temperature)) of each row; 0, 0 where no entry is kept."""
    s = logits.float()
    top = s.amax(1)
    total = torch.exp((s - top[:, None]) / temperature).sum(1).log()
    some = _kept(index, teacher, logits.shape[1]).any(1)
    return torch.where(some[:, None], torch.stack([top, total], 1), 0.0)


def _teacher(s):
    """(log p, p, kept, index) of the teacher's entries; p is 0 at those not kept."""
    t, index = s["teacher"].float(), s["index"].long()
    kept = _kept(index, t, s["vocab"])
    t = torch.where(kept, t, -math.inf)
    top = t.amax(1, keepdim=True)
    t = (t - torch.where(top > -math.inf, top, 0.0)) / s["temperature"]
    logp = t - torch.exp(t).sum(1, keepdim=True).log()
    return logp, torch.where(kept, torch.exp(logp), 0.0), kept, torch.where(kept, index, 0)


def _plain_norm_fwd(s):
    dt = DT[s["dtype"]]
    x = s["x"].float()
    mean = x.mean(1)
    x = x - mean[:, None]
    rstd = torch.rsqrt(x.square().mean(1) + EPS)
    y = x * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(dt), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    dt, pt = DT[s["dtype"]], DT[s["params"]]
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(0).to(pt), "dbeta": dy.sum(0).to(pt)}


def _plain_linear_fwd(s):
    dt = DT[s["dtype"]]
    z = s["x"].float() @ s["w"].float().t() + s["bias"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(dt)} if s["z"] is None else {"y": y.to(dt), "z": z.to(dt)}


def _plain_linear_bwd(s):
    dt = DT[s["dtype"]]
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["act"])
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt), "dbias": dz.sum(0).to(dt)}


def _plain_distill_fwd(s):
    stats = _distill_stats(s["logits"], s["index"], s["teacher"], s["temperature"])
    logp, p, kept, index = _teacher(s)
    logq = (s["logits"].gather(1, index).float() - stats[:, :1]) / s["temperature"] - stats[:, 1:]
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(1) * s["temperature"] ** 2
    return {"loss": loss, "stats": stats}


def _plain_distill_bwd(s):
    _, p, kept, index = _teacher(s)
    scale = (s["dloss"] * s["temperature"])[:, None]
    q = torch.exp((s["logits"].float() - s["stats"][:, :1]) / s["temperature"] - s["stats"][:, 1:])
    d = torch.where(kept.any(1)[:, None], q, 0.0)
    d = d.scatter_add(1, index, -p) * scale
    return d.to(DT[s["dtype"]])


_PLAIN = {("norm", "fwd"): _plain_norm_fwd, ("norm", "bwd"): _plain_norm_bwd,
          ("linear", "fwd"): _plain_linear_fwd, ("linear", "bwd"): _plain_linear_bwd,
          ("distill", "fwd"): _plain_distill_fwd, ("distill", "bwd"): _plain_distill_bwd}


# ------------------------------------------------------------------ the framework's calls

def _scratch(s, size):
    """The workspace of a call, kept with the buffers from the first call on."""
    if "scratch" not in s:
        s["scratch"] = torch.empty(max(16, size()), device="cuda", dtype=torch.uint8)
    return s["scratch"]


def _own_norm_fwd(s, v):
    v.vrcclLayerNormForward(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], s["rows"], s["cols"],
                            s["dtype"], s["params"], EPS, ldx=s["cols"] + s["pad"], ldy=s["cols"] + s["pad"])
    return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_norm_bwd(s, v):
    ld = s["cols"] + s["pad"]
    ws = _scratch(s, lambda: v.vrcclLayerNormWorkspace(s["rows"], s["cols"]))
    v.vrcclLayerNormBackward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"],
                             s["rows"], s["cols"], s["dtype"], s["params"], ws, ws.numel(), lddy=ld, ldx=ld, lddx=ld)
    return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def _own_linear_fwd(s, v):
    ldi, ldo = s["ins"] + s["pad"], s["outs"] + s["pad"]
    ws = _scratch(s, lambda: v.vrcclLinearWorkspace("forward", s["rows"], s["outs"], s["ins"], s["dtype"], s["act"]))
    v.vrcclLinearForward(s["x"], s["w"], s["bias"], s["r"], s["y"], s["z"], s["rows"], s["outs"], s["ins"],
                         s["dtype"], s["act"], ws, ws.numel(), ldx=ldi, ldw=ldi, ldr=ldo, ldy=ldo, ldz=ldo)
    return {"y": s["y"]} if s["z"] is None else {"y": s["y"], "z": s["z"]}


def _own_linear_bwd(s, v):
    ldi, ldo = s["ins"] + s["pad"], s["outs"] + s["pad"]
    ws = _scratch(s, lambda: v.vrcclLinearWorkspace("backward", s["rows"], s["outs"], s["ins"], s["dtype"], s["act"]))
    v.vrcclLinearBackward(s["dy"], s["z"], s["x"], s["w"], s["dx"], s["dw"], s["dbias"], s["rows"], s["outs"],
                          s["ins"], s["dtype"], s["act"], ws, ws.numel(), lddy=ldo, ldz=ldo, ldx=ldi, ldw=ldi,
                          lddx=ldi, lddw=ldi)
    return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}


def _own_distill_fwd(s, v):
    v.vrcclDistillForward(s["logits"], s["teacher"], s["index"], s["loss"], s["stats"], s["rows"], s["vocab"],
                          s["k"], s["dtype"], s["dtype"], s["index"].dtype, s["temperature"],
                          ldl=s["vocab"] + s["pad"])
    return {"loss": s["loss"], "stats": s["stats"]}


def _own_distill_bwd(s, v):
    ld = s["vocab"] + s["pad"]
    v.vrcclDistillBackward(s["logits"], s["teacher"], s["index"], s["stats"], s["dloss"], s["dlogits"], s["rows"],
                           s["vocab"], s["k"], s["dtype"], s["dtype"], s["index"].dtype, s["temperature"],
                           ldl=ld, ldd=ld)
    return s["dlogits"]


_OWN = {("norm", "fwd"): _own_norm_fwd, ("norm", "bwd"): _own_norm_bwd,
        ("linear", "fwd"): _own_linear_fwd, ("linear", "bwd"): _own_linear_bwd,
        ("distill", "fwd"): _own_distill_fwd, ("distill", "bwd"): _own_distill_bwd}


def run(s):
    if own:
        from ring_allreduce_reduction_gb300 import vrccl
        return _OWN[s["op"], s["dir"]](s, vrccl)
    return _PLAIN[s["op"], s["dir"]](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "norm":
        n, w, pe = c["rows"], c["cols"], SIZE[c["params"]]
        if c["dir"] == "fwd":
            return {"bytes": 2 * n * w * e + 8 * n + 2 * w * pe, "flops": 8 * n * w}
        return {"bytes": 3 * n * w * e + 8 * n + 3 * w * pe, "flops": 14 * n * w}
    if c["op"] == "linear":
        m, o, i, act = c["rows"], c["outs"], c["ins"], c["act"] != "none"
        if c["dir"] == "fwd":
            return {"bytes": e * (m * i + o * i + o + m * o * (1 + act + c["residual"])), "flops": 2 * m * o * i}
        return {"bytes": e * (m * o * (1 + act) + 2 * m * i + 2 * o * i + o), "flops": 4 * m * o * i}
    n, v, k = c["rows"], c["vocab"], c["k"]
    entries = n * k * (e + (4 if c["index"] == "int32" else 8))
    rows = n * (1 - c["empty"])  # positions without entries need no logits read
    if c["dir"] == "fwd":
        return {"bytes": int(rows * v * e) + entries + 12 * n, "flops": 4 * n * v}
    return {"bytes": int((rows + n) * v * e) + entries + 12 * n, "flops": 5 * n * v}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(s):
    x, gamma, beta = s["x"], s["gamma"].double().requires_grad_(), s["beta"].double().requires_grad_()
    out = []
    for at in range(0, s["rows"], 4096):
        part = x[at:at + 4096].double().requires_grad_()
        var, mean = torch.var_mean(part, 1, correction=0, keepdim=True)
        y = (part - mean) / torch.sqrt(var + EPS) * gamma + beta
        if s["dir"] == "fwd":
            out.append([t.detach() for t in (y, mean[:, 0], (var[:, 0] + EPS) ** -0.5)])
        else:
            y.backward(s["dy"][at:at + 4096].double())
            out.append([part.grad])
    if s["dir"] == "fwd":
        return dict(zip(("y", "mean", "rstd"), (torch.cat(t) for t in zip(*out))))
    return {"dx": torch.cat([t[0] for t in out]), "dgamma": gamma.grad, "dbeta": beta.grad}


def _exact_act(z, act):
    F = torch.nn.functional
    return {"none": lambda t: t, "relu": F.relu, "gelu": F.gelu, "gelu_tanh": lambda t: F.gelu(t, approximate="tanh"),
            "silu": F.silu}[act](z)


def _exact_linear(s):
    x, w = s["x"].double(), s["w"].double()
    if s["dir"] == "fwd":
        z = torch.addmm(s["bias"].double(), x, w.t())
        y = _exact_act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].double()
        return {"y": y} if s["z"] is None else {"y": y, "z": z}
    dz = s["dy"].double()
    if s["z"] is not None:
        z = s["z"].double().requires_grad_()
        dz, = torch.autograd.grad(_exact_act(z, s["act"]), z, dz)
    return {"dx": torch.mm(dz, w), "dw": torch.mm(dz.t(), x), "dbias": dz.sum(0)}


def _exact_distill(s):
    T, out = s["temperature"], []
    for at in range(0, s["rows"], 256):
        rows = slice(at, at + 256)
        logits = s["logits"][rows].double().requires_grad_()
        index, teacher = s["index"][rows].long(), s["teacher"][rows].double()
        kept = _kept(index, teacher, s["vocab"])
        some = kept.any(1)
        p = torch.softmax(torch.where(kept, teacher / T, -math.inf), 1).nan_to_num(0.0)
        logq = torch.log_softmax(logits / T, 1)
        terms = torch.special.xlogy(p, p) - p * logq.gather(1, index.clamp(0, s["vocab"] - 1))
        loss = T * T * terms.sum(1)
        if s["dir"] == "bwd":
            out.append(torch.autograd.grad(loss, logits, s["dloss"][rows].double())[0])
        else:
            top = logits.detach().amax(1)
            total = torch.logsumexp(logits.detach() / T, 1) - top / T
            out.append([loss.detach(), torch.where(some[:, None], torch.stack([top, total], 1), 0.0)])
    if s["dir"] == "bwd":
        return torch.cat(out)
    return dict(zip(("loss", "stats"), (torch.cat(t) for t in zip(*out))))


def exact(case, seed):
    return {"norm": _exact_norm, "linear": _exact_linear, "distill": _exact_distill}[case["op"]](prepare(case, seed))
