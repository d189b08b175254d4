"""The tensor functions record no graph (CPU only: refused before the device is looked at): a tensor
that requires a gradient is refused where one would be lost without a word."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z
from zero_partitioned_mixed_flat_gb300 import _abi as A
from zero_partitioned_mixed_flat_gb300 import head

X = torch.zeros(4, 64, dtype=torch.bfloat16)
W = torch.zeros(64, dtype=torch.bfloat16)
V = torch.zeros(10, 64, dtype=torch.bfloat16)
Y = torch.zeros(4, dtype=torch.int64)
F = torch.zeros(4)


def grown(t):
    return t.clone().requires_grad_()


CALLS = [
    lambda g: Z.residual_norm(g(X), None, W, 1e-5), lambda g: Z.residual_norm(X, g(X), W, 1e-5),
    lambda g: Z.residual_norm(X, None, g(W), 1e-5), lambda g: Z.residual_norm_quantized(g(X), None, W, 1e-5),
    lambda g: Z.residual_norm_backward(X, g(W), X, None, 1e-5), lambda g: Z.residual_norm_backward(X, W, X, g(X), 1e-5),
    lambda g: Z.linear_loss(g(X), V, Y), lambda g: Z.linear_loss(X, g(V), Y),
    lambda g: Z.linear_loss_backward(X, g(V), Y, F, F), lambda g: Z.linear_loss_backward(X, V, Y, F, g(F)),
]


@pytest.fixture(autouse=True)
def a_device(monkeypatch):
    """The CPU stands for the current device; nothing is launched: a call that gets further asks for the library."""
    def reached(*args):
        raise LookupError
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(head, "_call", reached)
    monkeypatch.setattr(head, "_status", lambda device: F)
    monkeypatch.setattr(A, "_stream", lambda stream: 0)


@pytest.mark.parametrize("call", CALLS)
def test_tensors_that_require_gradients_are_refused(call):
    with pytest.raises(Z.ZeroError, match="requires grad") as e:
        call(grown)
    assert e.value.code == Z.ZERO_EINVAL


@pytest.mark.parametrize("call", CALLS)
def test_detached_or_under_no_grad_they_are_taken(call):
    with pytest.raises(LookupError):
        call(lambda t: grown(t).detach())
    with torch.no_grad(), pytest.raises(LookupError):
        call(grown)
