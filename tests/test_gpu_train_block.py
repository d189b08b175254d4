"""The operators of a training step in a row, as train_head runs them with a gated block: norm, gated projections, norm,
loss, their gradients, the gradients' norm, and the step over tensors."""
import math

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z
from zero_partitioned_mixed_flat_gb300 import train_head

pytestmark = pytest.mark.gpu
HALF = torch.finfo(torch.bfloat16).eps / 2


def loss64(weights, tokens, targets):
    last, before, scale, matrix, gate, up, down, second = weights
    total = last[tokens[:, 1]] + before[tokens[:, 0]]
    norm = lambda t, w: t * (t.square().mean(1, keepdim=True) + train_head.EPS).rsqrt() * w  # noqa: E731
    hidden = norm(total, scale)
    a = hidden @ gate.T
    total = total + (a * torch.sigmoid(a) * (hidden @ up.T)) @ down.T
    z = norm(total, second) @ matrix.T
    counted = targets != train_head.IGNORE
    return torch.nn.functional.cross_entropy(z[counted], targets[counted])


def setup(vocab=72, dim=64, wide=136, tokens=500, key=0):
    gen = torch.Generator(device="cuda").manual_seed(key)
    model = train_head.BigramHead(vocab, dim, wide)
    weights = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in model.shapes]
    train_head.start(model, weights, gen)
    successors = torch.stack([torch.randperm(vocab, generator=gen, device="cuda") for _ in range(2)])
    return model, weights, train_head.batch(successors, tokens, gen)


def test_gradients_of_the_chain():
    """Each tensor's gradient within what the bf16 stages can add up to: at most sixteen roundings lie on the way from
    a weight to its gradient (norms, projections, products and their gradients), independent of each other and each
    off by half a step at most of a term, so the error's 2-norm is below 16 half steps of the gradient's; the loss below
    16 half steps of the logits' spread."""
    model, weights, (tokens, targets) = setup()
    loss, grads = model.gradients(weights, tokens, targets, int((targets != train_head.IGNORE).sum()))
    leaves = [w.double().requires_grad_() for w in weights]
    want = loss64(leaves, tokens, targets)
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 16 * HALF * 8
    for g, w, leaf in zip(grads, weights, leaves):
        assert g.shape == w.shape
        off = (g.double() - leaf.grad).norm() / leaf.grad.norm()
        assert off <= 16 * HALF, float(off)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_over_the_chains_weights(bits):
    """Two clipped steps follow the formula from the very gradients that the model gave (32 bits: to float rounding; 8
    bits: the second step's moments are off by the first's rounding, a sixteenth of m and a thirty-second of the root)."""
    model, weights, (tokens, targets) = setup(key=1)
    master = [w.float() for w in weights]
    state = Z.adamw_state(master, bits)
    m, v, p = ([torch.zeros_like(w, dtype=torch.float64) for w in weights] for _ in range(3))
    for i, w in enumerate(master):
        p[i] = w.double()
    lr = 1e-2
    for t in (1, 2):
        loss, grads = model.gradients(weights, tokens, targets, 100)
        norm, coef, bad = Z.gradient_norm(grads, 0.5)
        total = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        assert abs(float(norm) - total) <= 1e-5 * total and abs(float(coef) - min(1, 0.5 / (total + 1e-6))) <= 1e-5
        Z.adamw_step(master, grads, state, lr, 0.9, 0.99, 1e-8, 0.1, copies=weights, coef=coef, skip=bad)
        for i, g in enumerate(grads):
            f = g.double() * float(coef)
            m[i], v[i] = 0.9 * m[i] + 0.1 * f, 0.99 * v[i] + 0.01 * f * f
            p[i] = p[i] * (1 - lr * 0.1) - lr * (m[i] / (1 - 0.9 ** t)) / ((v[i] / (1 - 0.99 ** t)).sqrt() + 1e-8)
            slack = 1e-5 if bits == 32 or t == 1 else 0.15
            assert ((master[i].double() - p[i]).abs() <= 2e-6 * p[i].abs() + slack * lr).all()
            assert torch.equal(weights[i], master[i].to(torch.bfloat16))
            p[i] = master[i].double()   # the next gradients are those of the weights as they are
    assert int(state.record[0]) == 2
    Z.check_losses()


@pytest.mark.parametrize("call", [lambda: train_head.train(steps=3, ranks=2, wide=64, tokens=256),
                                  lambda: train_head.train_whole(steps=3, wide=64, tokens=256, bits=8),
                                  lambda: train_head.train_whole(steps=3, tokens=256)])
def test_the_example_runs(call):
    losses = call()
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)
