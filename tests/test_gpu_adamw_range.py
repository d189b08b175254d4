"""The ends of the range of the step with 8-bit moments: what it updates with is the 32-bit step's, before it is rounded."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

from .test_gpu_adamw import BLOCK, HYPER, U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** 64, 1e25, -3.4e38])
@pytest.mark.parametrize("at", [0, 130, 299, 2000])
def test_a_gradient_whose_square_is_infinite(size, at):
    """Finite, but v is not: the root is infinite and the update 0, so the element only decays, with 32-bit moments and with
    8-bit ones alike; the others of its block are updated as ever.  What the block's scale holds afterwards is NaN."""
    n = 2500
    gen = torch.Generator(device="cuda").manual_seed(at)
    start = torch.randn(n, generator=gen, device="cuda")
    grad = torch.randn(n, generator=gen, device="cuda") * 1e-2
    grad[at] = size
    after, copies, states = [], [], []
    for bits in (32, 8):
        p, copy = start.clone(), torch.empty(n, device="cuda", dtype=torch.bfloat16)
        state = Z.adamw_state([p], bits)
        Z.adamw_step([p], [grad], state, copies=[copy], **{**HYPER, "beta2": 0.0})   # v is the square itself
        after.append(p)
        copies.append(copy)
        states.append(state)
    decayed = torch.tensor(1 - HYPER["lr"] * HYPER["weight_decay"], dtype=torch.float64).float().cuda() * start[at]
    assert all(torch.equal(p[at], decayed) for p in after)
    assert all(torch.equal(c, p.bfloat16()) for c, p in zip(copies, after))
    # the same root and moment; lr / c1 and the root of c2 rounded once more, an approximate quotient: 2^-20 of the update
    update = (after[0] - start).abs().double() + HYPER["lr"] * HYPER["weight_decay"] * start.abs().double()
    off = 2.0 ** -20 * update + 8 * U * start.abs().double()
    assert ((after[0].double() - after[1].double()).abs() <= off).all()
    blocks = torch.arange(states[1].v_scales.numel(), device="cuda") == at // BLOCK
    assert torch.equal(torch.isnan(states[1].v_scales), blocks)
    assert torch.isfinite(states[1].m_scales).all()
    assert (states[1].v[:-(-n // BLOCK) * BLOCK].view(-1, BLOCK)[blocks] == 0).all()
