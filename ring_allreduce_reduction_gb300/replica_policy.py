"""Data-parallel training on the log probabilities of given tokens, over the
virtual ranks of one GPU.

Every rank is a replica of a small pre-norm block and its head on a batch of
its own:

    h = rms(x)                           vrcclRmsNormForward
    b = silu(h W1^T + c1) W2^T           vrcclLinearForward, twice
    s = x + dropout(b)                   vrcclDropoutForward
    l = rms(s) W3^T                      vrcclRmsNormForward, vrcclLinearForward
    log probability of a token, entropy  vrcclLogProbForward

The objective is the mean of weight * log probability + bonus * entropy: with
weights of 1 a language model's, with advantages a policy gradient's; a token
outside the vocabulary is padding. A step is captured in one CUDA graph: all
ranks forward and backward, their gradients landing in one bf16 bucket a rank,
and the buckets' average by vrcclAllReduce. The dropout's seed is a word on the
GPU that the host changes between steps; a rank's rows are numbered from its
place in the whole batch, so that replicas draw masks of their own.

    python -m ring_allreduce_reduction_gb300.replica_policy --ranks 4 --steps 20
"""
from __future__ import annotations

import argparse

import torch

from . import vrccl as v
from .replica_step import DT, Bucket

EPS = 1e-5


def _layout(width: int, hidden: int, vocab: int) -> dict[str, tuple[int, ...]]:
    return {"g1": (width,), "w1": (hidden, width), "c1": (hidden,), "w2": (width, hidden), "g2": (width,),
            "w3": (vocab, width)}


class Replica:
    """One virtual rank: its batch, activations, gradients and scratch."""

    def __init__(self, rank: int, tokens: int, width: int, hidden: int, vocab: int, p: float, bonus: float, seed):
        self.n, self.w, self.h, self.vocab, self.p, self.first = tokens, width, hidden, vocab, p, rank * tokens
        self.seed = seed  # the step's, on the GPU
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device="cuda")  # noqa: E731
        self.x, self.token, self.weight = bf(tokens, width), torch.empty(tokens, dtype=torch.int64, device="cuda"), f32(tokens)
        self.h1, self.b, self.s, self.h2 = (bf(tokens, width) for _ in range(4))
        self.z, self.a, self.logits = bf(tokens, hidden), bf(tokens, hidden), bf(tokens, vocab)
        self.r1, self.r2, self.logprob, self.entropy, self.stats = f32(tokens), f32(tokens), f32(tokens), f32(tokens), f32(tokens, 2)
        self.dlogprob, self.dentropy = f32(tokens), torch.full((1,), -bonus / tokens, device="cuda")
        self.dh, self.ds, self.db, self.da, self.dx = bf(tokens, width), bf(tokens, width), bf(tokens, width), bf(tokens, hidden), bf(tokens, width)
        self.grad = Bucket(_layout(width, hidden, vocab))
        need = [v.vrcclRmsNormWorkspace(tokens, width)]
        for outs, ins, act in ((hidden, width, "silu"), (width, hidden, "none"), (vocab, width, "none")):
            need += [v.vrcclLinearWorkspace(d, tokens, outs, ins, DT, act) for d in ("forward", "backward")]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")

    def load(self, x, token, weight) -> None:
        self.x.copy_(x)
        self.token.copy_(token)
        self.weight.copy_(weight)

    def forward(self, p: Bucket) -> None:
        n, w, ws = self.n, self.w, (self.ws, self.ws.numel())
        v.vrcclRmsNormForward(self.x, None, p["g1"], None, self.h1, self.r1, n, w, DT, DT, EPS)
        v.vrcclLinearForward(self.h1, p["w1"], p["c1"], None, self.a, self.z, n, self.h, w, DT, "silu", *ws)
        v.vrcclLinearForward(self.a, p["w2"], None, None, self.b, None, n, w, self.h, DT, "none", *ws)
        v.vrcclDropoutForward(self.b, self.x, self.s, n, w, DT, self.p, self.seed, 0, self.first)
        v.vrcclRmsNormForward(self.s, None, p["g2"], None, self.h2, self.r2, n, w, DT, DT, EPS)
        v.vrcclLinearForward(self.h2, p["w3"], None, None, self.logits, None, n, self.vocab, w, DT, "none", *ws)
        v.vrcclLogProbForward(self.logits, self.token, self.logprob, self.entropy, self.stats, None, None, n, self.vocab, 0,
                              DT, "int64")

    def backward(self, p: Bucket) -> None:
        n, w, g, ws = self.n, self.w, self.grad, (self.ws, self.ws.numel())
        torch.mul(self.weight, -1.0 / n, out=self.dlogprob)
        # the gradient of minus the objective, in the logits' place
        v.vrcclLogProbBackward(self.logits, self.token, self.stats, self.entropy, self.dlogprob, self.dentropy, self.logits, n,
                               self.vocab, DT, "int64", dentropy_stride=0)
        v.vrcclLinearBackward(self.logits, None, self.h2, p["w3"], self.dh, g["w3"], None, n, self.vocab, w, DT, "none", *ws)
        v.vrcclRmsNormBackward(self.dh, None, self.s, p["g2"], self.r2, self.ds, g["g2"], n, w, DT, DT, *ws)
        v.vrcclDropoutBackward(self.ds, self.db, n, w, DT, self.p, self.seed, 0, self.first)
        v.vrcclLinearBackward(self.db, None, self.a, p["w2"], self.da, g["w2"], None, n, w, self.h, DT, "none", *ws)
        v.vrcclLinearBackward(self.da, self.z, self.h1, p["w1"], self.dh, g["w1"], g["c1"], n, self.h, w, DT, "silu", *ws)
        v.vrcclRmsNormBackward(self.dh, self.ds, self.x, p["g1"], self.r1, self.dx, g["g1"], n, w, DT, DT, *ws)

    def value(self) -> torch.Tensor:
        """The objective's mean over the rank's tokens."""
        return (self.weight * self.logprob).mean() - self.dentropy[0] * self.entropy.sum()


class Step:
    """All ranks' step; `run` takes it, from the second time on as a graph."""

    def __init__(self, ranks: int, tokens: int, width: int, hidden: int, vocab: int, p: float = 0.1, bonus: float = 0.01, seed: int = 0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.params = Bucket(_layout(width, hidden, vocab))
        for name, t in self.params.t.items():
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda") / t.shape[1] ** 0.5 if name[0] == "w" else torch.full_like(t, name[0] == "g"))
        self.seed = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.replicas = [Replica(r, tokens, width, hidden, vocab, p, bonus, self.seed) for r in range(ranks)]
        self.comm = v.vrcclCommInit(ranks, 8)
        self.graph = None

    def once(self) -> None:
        for rep in self.replicas:
            rep.forward(self.params)
            rep.backward(self.params)
        flats = [rep.grad.flat for rep in self.replicas]
        v.vrcclAllReduce(flats, flats, flats[0].numel(), DT, "avg", "auto", "auto", self.comm)

    def run(self, seed: int) -> None:
        self.seed.fill_(seed)
        if self.graph is None:
            self.once()
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.once()
        else:
            self.graph.replay()

    def check(self) -> None:
        torch.cuda.synchronize()
        for code in (v.vrcclCommGetAsyncError(self.comm), v.vrcclReplicaGetAsyncError()):
            v._check(code, "replica_policy")

    def close(self) -> None:
        self.graph = None
        v.vrcclCommDestroy(self.comm)


def batch(tokens: int, width: int, vocab: int, rank: int, seed: int = 1):
    """(x, tokens, weights) of a rank: each token's row points to it; a twelfth of them is padding."""
    gen = torch.Generator("cuda").manual_seed(seed)
    table = torch.randn(vocab, width, generator=gen, device="cuda")
    gen.manual_seed(seed + 1 + rank)
    token = (torch.rand(tokens, generator=gen, device="cuda") * vocab).long().clamp_(0, vocab - 1)
    x = (table[token] + torch.randn(tokens, width, generator=gen, device="cuda")).bfloat16()
    token[::12] = -1
    return x, token, 0.5 + torch.rand(tokens, generator=gen, device="cuda")


def train(ranks: int, tokens: int, width: int, hidden: int, vocab: int, steps: int, lr: float = 0.5) -> list[float]:
    """Runs the steps; returns the objective's mean over the ranks at each."""
    step, values = Step(ranks, tokens, width, hidden, vocab), []
    try:
        for r, rep in enumerate(step.replicas):
            rep.load(*batch(tokens, width, vocab, r))
        master = step.params.flat.float()
        for i in range(steps):
            step.run(i)
            values.append(torch.stack([rep.value() for rep in step.replicas]).mean())
            master.sub_(lr * step.replicas[0].grad.flat.float())
            step.params.flat.copy_(master)
        step.check()
    finally:
        step.close()
    return [x.item() for x in values]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("ranks", 4), ("tokens", 256), ("width", 256), ("hidden", 1024), ("vocab", 4096), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=default)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    for i, x in enumerate(train(a.ranks, a.tokens, a.width, a.hidden, a.vocab, a.steps, a.lr)):
        print(f"step {i:3d}  objective {x:.4f}")


if __name__ == "__main__":
    main()
