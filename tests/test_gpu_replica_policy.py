"""Dropout, RMS norm, linear layers, token log probabilities and the AllReduce
together: a data-parallel step's gradients against the same step in 64 bits,
and its captured form."""
import numpy as np
import pytest

from oracle import replica as o

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def policy():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_reduction_gb300 import build
    build.build()
    from ring_allreduce_reduction_gb300 import replica_policy
    return replica_policy


# activations and gradients are rounded to bf16 (by at most 2^-8 of themselves) some twelve times between a weight and the
# objective and back, once a rank in the average
BOUND = 14 * 2.0 ** -8


def _value64(torch, w, reps, kept, scale, bonus):
    """Mean over the ranks of the objective, in float64."""
    rms = lambda x, g: x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * g  # noqa: E731
    total = 0.0
    for rep, keep in zip(reps, kept):
        x = rep.x.double()
        b = torch.nn.functional.silu(rms(x, w["g1"]) @ w["w1"].t() + w["c1"]) @ w["w2"].t()
        s = x + torch.where(keep, b * scale, 0.0)
        logq = torch.log_softmax(rms(s, w["g2"]) @ w["w3"].t(), 1)
        given = rep.token >= 0
        logprob = logq.gather(1, rep.token.clamp(min=0)[:, None])[:, 0]
        entropy = -(logq.exp() * logq).sum(1)
        total = total + torch.where(given, rep.weight.double() * logprob + bonus * entropy, 0.0).mean() / len(reps)
    return total


@pytest.mark.parametrize("ranks,tokens,width,hidden,vocab", [(3, 96, 128, 512, 1000), (2, 33, 72, 200, 777)])
def test_step_against_64_bits(policy, ranks, tokens, width, hidden, vocab):
    """Eager, and replayed with another seed of the masks."""
    import torch
    p, bonus = 0.2, 0.05
    step = policy.Step(ranks, tokens, width, hidden, vocab, p, bonus)
    try:
        for r, rep in enumerate(step.replicas):
            rep.load(*policy.batch(tokens, width, vocab, r))
        grads = {}
        for seed in (11, 12, 11):
            step.run(seed)
            step.check()
            kept, scale = o.dropout_mask(ranks * tokens, width, p, seed, 0, 0)
            kept = torch.as_tensor(kept).cuda().view(ranks, tokens, width)
            w = {n: t.double().requires_grad_() for n, t in step.params.t.items()}
            value = _value64(torch, w, step.replicas, kept, scale, bonus)
            (-value).backward()
            got = torch.stack([rep.value() for rep in step.replicas]).mean().item()
            assert abs(got - value.item()) <= BOUND * abs(value.item())
            for rep in step.replicas:
                assert torch.equal(rep.grad.flat, step.replicas[0].grad.flat)  # every rank holds the average
            for name, t in w.items():
                g = step.replicas[0].grad[name].double()
                assert (g - t.grad).norm() <= BOUND * t.grad.norm(), (seed, name)
            # the same masks, the same bits, captured or not
            assert torch.equal(step.replicas[0].grad.flat, grads.setdefault(seed, step.replicas[0].grad.flat.clone()))
    finally:
        step.close()


def test_training_runs(policy):
    values = policy.train(2, 48, 64, 128, 300, steps=3)
    assert len(values) == 3 and np.isfinite(values).all()
