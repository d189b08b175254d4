"""The ends of the range of the step with 8-bit moments: what it updates with is the 32-bit step's, before it is rounded."""
import math

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

from .test_gpu_adamw import BLOCK, HYPER, U, codes_of, random16, values

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


@pytest.mark.parametrize("size", [1e-15, 1e-17, 1e-18, 1e-19, 1e-20, 3e-21])
@pytest.mark.parametrize("beta2", [0.999, 0.5])
def test_roots_of_the_smallest_squares(size, beta2):
    """v around and below 2^-126: the codes, the scales and, with an eps of 0, the updates of the float square root."""
    n, beta1, lr, seed = 1 << 14, 0.9, 1e-3, 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    p = torch.randn(n, generator=gen, device="cuda")
    state = Z.adamw_state([p], 8)
    for step in range(1, 4):
        g = (torch.rand(n, generator=gen, device="cuda") + 1) * size * (torch.randint(0, 2, (n,), generator=gen, device="cuda") * 2 - 1)
        m0, r0, _, _ = (x.float() for x in values(state))
        m = m0 * beta1 + g * (1 - beta1)
        r = ((r0 * r0) * beta2 + (g * g) * (1 - beta2)).sqrt()
        assert (r > 0).all()
        before = p.double()
        Z.adamw_step([p], [g], state, lr, beta1, beta2, 0.0, seed=seed)
        update = lr / (1 - beta1 ** step) * m.double() / (r.double() / math.sqrt(1 - beta2 ** step))
        # the constants of the corrections rounded to float, an approximate quotient, and the sum
        off = 2.0 ** -20 * update.abs() + 2 * U * (before.abs() + p.double().abs())
        assert ((p.double() - (before - update)).abs() <= off).all()
        bits_m, bits_r = random16(0, n, step, seed)
        code_m, scale_m = codes_of(m.abs(), 448.0, bits_m, 3, -6, 126)
        code_r, scale_r = codes_of(r, 1.96875 / 256, bits_r, 5, -14, 255)
        _, _, got_m, got_r = values(state)
        assert torch.equal(state.m_scales, scale_m) and torch.equal(state.v_scales, scale_r)
        assert torch.equal(got_m, code_m.long()) and torch.equal(got_r, code_r.clamp(min=1).long())


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-12, 1e-8])
def test_roots_of_squares_of_all_sizes(eps):
    """Gradients from 1e-20 to 1e3 in one block, and blocks of all sizes: the same, whatever the block's largest root."""
    n, beta1, beta2, lr, seed = 1 << 16, 0.9, 0.999, 1e-3, 9
    gen = torch.Generator(device="cuda").manual_seed(6)
    p = torch.randn(n, generator=gen, device="cuda")
    state = Z.adamw_state([p], 8)
    sign = torch.randint(0, 2, (n,), generator=gen, device="cuda") * 2 - 1
    block = torch.rand(n // BLOCK, generator=gen, device="cuda").mul_(23).repeat_interleave(BLOCK)
    for step in range(1, 4):
        size = torch.minimum(torch.rand(n, generator=gen, device="cuda").mul_(23), block)
        g = sign * 10.0 ** (size - 20)
        m0, r0, _, _ = (x.float() for x in values(state))
        m = m0 * beta1 + g * (1 - beta1)
        r = ((r0 * r0) * beta2 + (g * g) * (1 - beta2)).sqrt()
        assert (r > 0).all()
        before = p.double()
        Z.adamw_step([p], [g], state, lr, beta1, beta2, eps, seed=seed)
        update = lr / (1 - beta1 ** step) * m.double() / (r.double() / math.sqrt(1 - beta2 ** step) + eps)
        off = 2.0 ** -20 * update.abs() + 2 * U * (before.abs() + p.double().abs())
        assert ((p.double() - (before - update)).abs() <= off).all()
        bits_m, bits_r = random16(0, n, step, seed)
        code_m, scale_m = codes_of(m.abs(), 448.0, bits_m, 3, -6, 126)
        code_r, scale_r = codes_of(r, 1.96875 / 256, bits_r, 5, -14, 255)
        _, _, got_m, got_r = values(state)
        assert torch.equal(state.m_scales, scale_m) and torch.equal(state.v_scales, scale_r)
        assert torch.equal(got_m, code_m.long()) and torch.equal(got_r, code_r.clamp(min=1).long())
