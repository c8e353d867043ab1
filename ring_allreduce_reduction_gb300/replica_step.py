"""Data-parallel training by distillation over the virtual ranks of one GPU.

Every rank is a replica of a small head on a batch of its own:

    h = norm(x)                        vrcclLayerNormForward
    a = gelu(h W1^T + c1)              vrcclLinearForward (keeps z)
    y = a W2^T + c2 + x                vrcclLinearForward (residual)
    l = norm(y) W3^T                   vrcclLayerNormForward, vrcclLinearForward
    loss of l against the teacher's top logits   vrcclDistillForward

A step runs each replica forward and backward, its gradients landing in one
bf16 bucket a rank, averages the buckets with vrcclAllReduce, and applies
plain gradient descent to the weights the ranks share (held in binary32, where
a step of less than a bf16 unit is not lost, and rounded to bf16 for use).

    python -m ring_allreduce_reduction_gb300.replica_step --ranks 4 --steps 20
"""
from __future__ import annotations

import argparse

import torch

from . import vrccl as v

DT = "bfloat16"


def _layout(width: int, hidden: int, vocab: int) -> dict[str, tuple[int, ...]]:
    return {"g1": (width,), "b1": (width,), "w1": (hidden, width), "c1": (hidden,), "w2": (width, hidden),
            "c2": (width,), "g2": (width,), "b2": (width,), "w3": (vocab, width)}


class Bucket:
    """Named tensors in one flat bf16 buffer, each on a 16-byte boundary."""

    def __init__(self, shapes: dict[str, tuple[int, ...]], device="cuda"):
        at, places = 0, {}
        for name, shape in shapes.items():
            n = torch.Size(shape).numel()
            places[name] = (at, n, shape)
            at += (n + 7) // 8 * 8
        self.flat = torch.zeros(at, dtype=torch.bfloat16, device=device)
        self.t = {name: self.flat[a:a + n].view(shape) for name, (a, n, shape) in places.items()}

    def __getitem__(self, name: str) -> torch.Tensor:
        return self.t[name]


class Replica:
    """One virtual rank: its activations, gradients and scratch."""

    def __init__(self, tokens: int, width: int, hidden: int, vocab: int, k: int):
        self.n, self.w, self.h, self.vocab, self.k = tokens, width, hidden, vocab, k
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device="cuda")  # noqa: E731
        self.h1, self.y, self.h2 = bf(tokens, width), bf(tokens, width), bf(tokens, width)
        self.z, self.a, self.logits = bf(tokens, hidden), bf(tokens, hidden), bf(tokens, vocab)
        self.m1, self.r1, self.m2, self.r2 = (f32(tokens) for _ in range(4))
        self.loss, self.stats = f32(tokens), f32(tokens, 2)
        self.dh, self.dy, self.da, self.dx = bf(tokens, width), bf(tokens, width), bf(tokens, hidden), bf(tokens, width)
        self.dloss = torch.full((1,), 1.0 / tokens, device="cuda")
        self.grad = Bucket(_layout(width, hidden, vocab))
        need = [v.vrcclLayerNormWorkspace(tokens, width)]
        for outs, ins, act in ((hidden, width, "gelu"), (width, hidden, "none"), (vocab, width, "none")):
            need += [v.vrcclLinearWorkspace(d, tokens, outs, ins, DT, act) for d in ("forward", "backward")]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")

    def forward(self, p: Bucket, x, teacher, index, temperature: float) -> torch.Tensor:
        n, w, ws = self.n, self.w, (self.ws, self.ws.numel())
        v.vrcclLayerNormForward(x, p["g1"], p["b1"], self.h1, self.m1, self.r1, n, w, DT, DT)
        v.vrcclLinearForward(self.h1, p["w1"], p["c1"], None, self.a, self.z, n, self.h, w, DT, "gelu", *ws)
        v.vrcclLinearForward(self.a, p["w2"], p["c2"], x, self.y, None, n, w, self.h, DT, "none", *ws)
        v.vrcclLayerNormForward(self.y, p["g2"], p["b2"], self.h2, self.m2, self.r2, n, w, DT, DT)
        v.vrcclLinearForward(self.h2, p["w3"], None, None, self.logits, None, n, self.vocab, w, DT, "none", *ws)
        v.vrcclDistillForward(self.logits, teacher, index, self.loss, self.stats, n, self.vocab, self.k, DT,
                              teacher.dtype, index.dtype, temperature)
        return self.loss

    def backward(self, p: Bucket, x, teacher, index, temperature: float) -> None:
        n, w, g, ws = self.n, self.w, self.grad, (self.ws, self.ws.numel())
        # the mean over the tokens; the gradient takes the logits' place
        v.vrcclDistillBackward(self.logits, teacher, index, self.stats, self.dloss, self.logits, n, self.vocab, self.k,
                               DT, teacher.dtype, index.dtype, temperature, dloss_stride=0)
        v.vrcclLinearBackward(self.logits, None, self.h2, p["w3"], self.dh, g["w3"], None, n, self.vocab, w, DT, "none",
                              *ws)
        v.vrcclLayerNormBackward(self.dh, self.y, p["g2"], self.m2, self.r2, self.dy, g["g2"], g["b2"], n, w, DT, DT, *ws)
        v.vrcclLinearBackward(self.dy, None, self.a, p["w2"], self.da, g["w2"], g["c2"], n, w, self.h, DT, "none", *ws)
        v.vrcclLinearBackward(self.da, self.z, self.h1, p["w1"], self.dh, g["w1"], g["c1"], n, self.h, w, DT, "gelu", *ws)
        v.vrcclLayerNormBackward(self.dh, x, p["g1"], self.m1, self.r1, self.dx, g["g1"], g["b1"], n, w, DT, DT, *ws)


def init_params(width: int, hidden: int, vocab: int, seed: int = 0) -> Bucket:
    gen = torch.Generator("cuda").manual_seed(seed)
    p = Bucket(_layout(width, hidden, vocab))
    for name, t in p.t.items():
        if name[0] == "w":
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda") / t.shape[1] ** 0.5)
        elif name[0] == "g":
            t.fill_(1.0)
    return p


def batch(tokens: int, width: int, vocab: int, k: int, rank: int, seed: int = 1):
    """(x, teacher logits, indices) of a rank: the teacher is a fixed random map of x."""
    gen = torch.Generator("cuda").manual_seed(seed)
    wt = torch.randn(vocab, width, generator=gen, device="cuda") * (2.0 / width ** 0.5)
    gen.manual_seed(seed + 1 + rank)
    x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
    teacher, index = (x.float() @ wt.t()).topk(k, 1)
    return x, teacher, index


def train(ranks: int, tokens: int, width: int, hidden: int, vocab: int, k: int, steps: int, lr: float = 0.5,
          temperature: float = 2.0, seed: int = 0):
    """Runs the steps; returns (mean loss per step, the replicas, the weights)."""
    p = init_params(width, hidden, vocab, seed)
    master = p.flat.float()
    reps = [Replica(tokens, width, hidden, vocab, k) for _ in range(ranks)]
    data = [batch(tokens, width, vocab, k, r, seed + 1) for r in range(ranks)]
    comm = v.vrcclCommInit(ranks, 8)
    losses = []
    try:
        for _ in range(steps):
            for rep, (x, teacher, index) in zip(reps, data):
                rep.forward(p, x, teacher, index, temperature)
                rep.backward(p, x, teacher, index, temperature)
            flats = [rep.grad.flat for rep in reps]
            v.vrcclAllReduce(flats, flats, flats[0].numel(), DT, "avg", "auto", "auto", comm)
            losses.append(torch.stack([rep.loss.mean() for rep in reps]).mean())
            master.sub_(lr * reps[0].grad.flat.float())
            p.flat.copy_(master)
        torch.cuda.synchronize()
        for code in (v.vrcclCommGetAsyncError(comm), v.vrcclReplicaGetAsyncError()):
            v._check(code, "replica_step")
    finally:
        v.vrcclCommDestroy(comm)
    return [x.item() for x in losses], reps, p


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("ranks", 4), ("tokens", 256), ("width", 256), ("hidden", 1024), ("vocab", 4096), ("k", 32),
                          ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=default)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    losses, _, _ = train(a.ranks, a.tokens, a.width, a.hidden, a.vocab, a.k, a.steps, a.lr)
    for i, x in enumerate(losses):
        print(f"step {i:3d}  loss {x:.4f}")


if __name__ == "__main__":
    main()
