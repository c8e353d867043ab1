"""The replica's operators and the AllReduce together: a data-parallel
distillation step against the same step in 64 bits, and a few steps of training."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def step():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_reduction_gb300 import build
    build.build()
    from ring_allreduce_reduction_gb300 import replica_step
    return replica_step


# activations and gradients are rounded to bf16 (by at most 2^-8 of themselves) some ten times between a weight and the
# loss and back, once a rank in the average
BOUND = 12 * 2.0 ** -8


def _loss64(w, data, temperature):
    """Mean over the ranks of the loss, in float64."""
    import torch
    F = torch.nn.functional
    total = 0.0
    for x, teacher, index in data:
        x = x.double()
        h = F.layer_norm(x, x.shape[1:], w["g1"], w["b1"])
        y = F.gelu(h @ w["w1"].t() + w["c1"]) @ w["w2"].t() + w["c2"] + x
        logits = F.layer_norm(y, x.shape[1:], w["g2"], w["b2"]) @ w["w3"].t()
        t = torch.log_softmax(teacher.double() / temperature, 1)
        q = torch.log_softmax(logits / temperature, 1).gather(1, index)
        total = total + ((t.exp() * (t - q)).sum(1) * temperature ** 2).mean() / len(data)
    return total


@pytest.mark.parametrize("ranks,tokens,width,hidden,vocab,k", [(4, 96, 128, 512, 1000, 16), (2, 33, 72, 200, 777, 5)])
def test_step_against_64_bits(step, ranks, tokens, width, hidden, vocab, k):
    import torch
    losses, reps, _ = step.train(ranks, tokens, width, hidden, vocab, k, steps=1, lr=0.0)
    data = [step.batch(tokens, width, vocab, k, r, 1) for r in range(ranks)]
    w = {n: t.double().requires_grad_() for n, t in step.init_params(width, hidden, vocab, 0).t.items()}
    loss = _loss64(w, data, 2.0)
    loss.backward()
    assert abs(losses[0] - loss.item()) <= BOUND * loss.item()
    for rep in reps:
        assert torch.equal(rep.grad.flat, reps[0].grad.flat)  # every rank holds the average
    for name, t in w.items():
        got = reps[0].grad[name].double()
        assert (got - t.grad).norm() <= BOUND * t.grad.norm(), name


def test_training_follows_64_bits(step):
    """Several steps of descent: the loss falls at each, as it does in 64 bits."""
    import torch
    shape = {"width": 128, "hidden": 256, "vocab": 1024}
    losses, _, _ = step.train(4, 128, k=16, steps=6, lr=0.5, **shape)
    data = [step.batch(128, 128, 1024, 16, r, 1) for r in range(4)]
    w = {n: t.double().requires_grad_() for n, t in step.init_params(**shape, seed=0).t.items()}
    for i, got in enumerate(losses):
        loss = _loss64(w, data, 2.0)
        assert abs(got - loss.item()) <= BOUND * loss.item()
        assert i == 0 or got < losses[i - 1]
        grads = torch.autograd.grad(loss, list(w.values()))
        w = {n: (t - 0.5 * g).detach().requires_grad_() for (n, t), g in zip(w.items(), grads)}
