"""What the calls on torch tensors write counts as written to autograd: a step between a forward pass and its backward
pass is an error there, as torch's own optimizers make it, and no silently wrong gradient."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def stepped(bits, master, copies, **more):
    grads = [torch.ones_like(m) for m in master]
    state = Z.adamw_state(master, bits)
    Z.adamw_step(master, grads, state, 1e-2, copies=copies, **more)
    return state, grads


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_between_forward_and_backward(bits):
    p = torch.nn.Parameter(torch.randn(300, device="cuda"))
    w = torch.nn.Parameter(p.detach().to(BF))
    for leaf in (p, w):
        loss = (leaf * leaf).sum()
        stepped(bits, [p], [w.detach()])
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    (w * w).sum().backward()
    assert torch.equal(w.grad, 2 * w.detach())


@pytest.mark.parametrize("bits", [32, 8])
def test_everything_written_and_nothing_else(bits):
    master, copies = [torch.zeros(n, device="cuda") for n in (130, 0, 7)], [torch.zeros(n, device="cuda", dtype=BF) for n in (130, 0, 7)]
    coef, skip = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda", dtype=torch.int32)
    state, grads = stepped(bits, master, copies, coef=coef, skip=skip)
    assert [t._version for t in (*master, *copies)] == [1] * 6
    assert [t._version for t in state if t is not None] == [1] * (3 if bits == 32 else 5)
    assert [t._version for t in (*grads, coef, skip)] == [0] * 5
    with pytest.raises(Z.ZeroError):
        Z.adamw_step(master, grads, state, float("nan"), copies=copies)
    assert [t._version for t in (*master, *copies)] == [1] * 6
    with torch.inference_mode():
        frozen = [torch.zeros(130, device="cuda")]
    stepped(bits, frozen, None)


def test_gradients_that_are_given():
    x, gate, up, grad = (torch.randn(n, m, device="cuda").to(BF) for n, m in ((4, 16), (24, 16), (24, 16), (4, 24)))
    into = torch.zeros(24, 16, device="cuda", dtype=BF)
    Z.gated_linear_backward(x, gate, up, grad, grad_up=into)
    assert into._version == 1 and [t._version for t in (x, gate, up, grad)] == [0] * 4
