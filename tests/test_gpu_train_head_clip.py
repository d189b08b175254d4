"""The example clips what a training step clips: the gradient averaged over the ranks, once."""
import math

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z
from zero_partitioned_mixed_flat_gb300 import train_head

pytestmark = pytest.mark.gpu


def one_step(monkeypatch, ranks, clip):
    """What one step of the example packs, for each rank its gradients and its flat buffer, and the step's result."""
    packed, results, hypers = [], [], []
    clip_gradients, hyper, result = train_head.clip_gradients, train_head.Hyper, Z.ZeroPlan.result

    def watched(grads, flat, offsets, **options):
        before = [g.clone() for g in grads]
        got = clip_gradients(grads, flat, offsets, **options)
        packed.append((torch.cat([g.flatten() for g in before]), flat.clone()))
        return got

    monkeypatch.setattr(train_head, "clip_gradients", watched)
    monkeypatch.setattr(train_head, "Hyper", lambda *a: hypers.append(hyper(*a)) or hypers[-1])
    monkeypatch.setattr(Z.ZeroPlan, "result", lambda plan: results.append(result(plan)) or results[-1])
    train_head.train(steps=1, ranks=ranks, vocab=32, dim=64, tokens=512, clip=clip)
    assert len(packed) == ranks and len(hypers) == 1
    return packed, hypers[0], results[-1]


@pytest.mark.parametrize("ranks", [1, 3])
def test_the_step_clips_the_averaged_gradient(monkeypatch, ranks):
    clip = 1e-3                                          # below every rank's norm
    packed, hyper, result = one_step(monkeypatch, ranks, clip)
    for grads, flat in packed:
        assert grads.double().norm() > 2 * clip
        assert torch.equal(flat[:grads.numel()], grads)  # as they are
    assert hyper.clip == clip
    mean = sum(flat.double() for _, flat in packed) / ranks
    # the norm's squares are float numbers added up in double: 2^-23 of each
    assert math.isclose(result["norm"], mean.norm().item(), rel_tol=2.0 ** -22)
