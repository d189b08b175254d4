"""The training head and the ZeRO step together: the example's gradients against
automatic differentiation in 64 bits, and its loss over some steps."""
import math

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z
from zero_partitioned_mixed_flat_gb300 import train_head

pytestmark = pytest.mark.gpu


def test_example_gradients():
    vocab, dim, n = 48, 72, 500
    gen = torch.Generator(device="cuda").manual_seed(4)
    model = train_head.BigramHead(vocab, dim)
    flat = torch.randn(sum(model.sizes), generator=gen, device="cuda").to(torch.bfloat16) * 0.3
    offsets = [0, vocab * dim, 2 * vocab * dim, 2 * vocab * dim + dim]
    weights = model.views(flat, offsets)
    tokens = torch.randint(0, vocab, (n, 2), generator=gen, device="cuda")
    targets = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    targets[::5] = train_head.IGNORE
    counted = int((targets >= 0).sum())
    loss, grads = model.gradients(weights, tokens, targets, counted)
    Z.check_losses()
    exact = [w.double().requires_grad_() for w in weights]
    s = exact[0][tokens[:, 1]] + exact[1][tokens[:, 0]]
    hidden = s * (s.square().mean(1, keepdim=True) + train_head.EPS).rsqrt() * exact[2]
    ref = torch.nn.functional.cross_entropy(hidden @ exact[3].t(), targets, ignore_index=train_head.IGNORE)
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 2.0 ** -7 * ref.item()
    for g, w in zip(grads, exact):
        # hidden, its gradient, the sum and the result are rounded to 8 bits on the way
        assert (g.double() - w.grad).norm() <= 4 * 2.0 ** -8 * w.grad.norm()


@pytest.mark.parametrize("ranks", [1, 3])
def test_example_learns(ranks):
    losses = train_head.train(steps=40, ranks=ranks, vocab=32, dim=64, tokens=1024)
    assert losses[0] < 2 * math.log(32) and all(math.isfinite(x) for x in losses)
    assert losses[-1] < losses[0] - 1.0
