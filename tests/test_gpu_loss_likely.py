"""Targets that are all but certain: their slope is what is left of a difference of nearly equal numbers."""
import math

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def batch(t, d, v, dtype, above):
    """Tokens whose target's logit stands `above` over the logarithm of all others' sum, a sum that grows evenly."""
    gen = torch.Generator(device="cuda").manual_seed(t + d)
    w = (0.05 * torch.randn(v, d, generator=gen, device="cuda")).to(dtype)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    high = math.log(v) + above
    wy = w[y].float()
    h = (0.2 * torch.randn(t, d, generator=gen, device="cuda") + high * wy / wy.square().sum(1, keepdim=True)).to(dtype)
    z = h.double() @ w.double().t()
    rest = z.clone()
    rest[torch.arange(t), y] = -math.inf
    at = z.gather(1, y[:, None])[:, 0]
    # 1 - p without the cancellation, and the loss: log(1 + e^x), x = what the others' sum is below the target
    x = torch.logsumexp(rest, 1) - at
    return h, w, y, torch.logsumexp(z, 1), torch.nn.functional.softplus(x), torch.sigmoid(x)


SHAPES = [(1, 4096, 500), (2, 768, 9000), (3, 536, 821), (5, 1024, 500), (40, 4096, 700), (300, 2056, 700), (700, 1600, 20000), (4100, 264, 3000)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("above", [4.6, 6.9, 9.2])
@pytest.mark.parametrize("t,d,v", SHAPES)
def test_targets_that_are_all_but_certain(t, d, v, dtype, above):
    """The slope is expm1(z - lse) with a float z that lse contains as well, so what z itself is off cancels.

    What is left of a slope: lse is a float, half of 2^-19 between 16 and 32, and as much again for its own arithmetic
    and for z - lse; and the others' exponentials, 1e-4 of it (their logits, at most 34 steps of 2^-22 of sums of
    magnitude 10 here, and 2e-6).  Besides, the slopes' and the result's rounding to 16 bits, each as large as e,
    that of the exact gradients.
    """
    h, w, y, ref_lse, ref_loss, missing = batch(t, d, v, dtype, above)
    slack = 2.0 ** -19
    loss, lse = Z.linear_loss(h, w, y)
    # z, up to 20, is a float sum in 32 lanes: d / 32 products each and five sums of lanes, half of 2^-23 of 20 at most
    z_off = (d / 32 + 5) * 2.0 ** -24 * 20
    assert ((lse.double() - ref_lse).abs() <= slack + z_off).all()
    assert ((loss.double() - ref_loss).abs() <= slack + ref_loss * 1e-4).all()
    gh, gw = Z.linear_loss_backward(h, w, y, lse, torch.ones(t, device="cuda"))
    Z.check_losses()
    q = torch.exp(h.double() @ w.double().t() - ref_lse[:, None])
    q[torch.arange(t), y] = -missing
    for got, ref in ((gh, q @ w.double()), (gw, q.t() @ h.double())):
        e = ((ref.to(dtype).double() - ref).norm() / ref.norm()).item()
        room = 2.1 * e + 1e-4 + slack * t ** 0.5 / missing.norm().item()
        err = ((got.double() - ref).norm() / ref.norm()).item()
        assert err <= room, (err, room)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [1024, 4096, 8200])
@pytest.mark.parametrize("t,v", [(200, 300), (700, 40000)])
def test_another_logit_that_is_all_of_lse(t, d, v, dtype):
    """One logit of 18 to 30 that is not the target's: the tensor core's sum, taken off after at most 512 products.

    Each 16 products drop less than 2^-23 of what the sum then is, and in fp16, whose products are longer, as much
    again as it aligns them: 32 steps, on average half as large as at the end, are 16.5 units of 2^-23, of 2^-22 in
    fp16.  Beside that the parts' additions and the rounding of lse, a few 2^-24 taken as 4, and the 4e-6 of the
    exponentials over at least 18.  (Of 4096 products in one sum the mean would be 5.5e-6 in bf16.)
    """
    gen = torch.Generator(device="cuda").manual_seed(d)
    w = (0.02 * torch.randn(v, d, generator=gen, device="cuda")).to(dtype)
    top = torch.randint(0, v, (t,), generator=gen, device="cuda")
    high = 18 + 12 * torch.rand(t, 1, generator=gen, device="cuda")
    h = (0.1 * torch.randn(t, d, generator=gen, device="cuda") + high * w[top].float() / (0.0004 * d)).to(dtype)
    y = (top + 1) % v
    loss, lse = Z.linear_loss(h, w, y)
    z = h.double() @ w.double().t()
    ref = torch.logsumexp(z, 1)
    room = 16.5 * 2.0 ** (-23 if dtype == BF else -22) + 4 * 2.0 ** -24 + 4e-6 / 18
    off = ((lse.double() - ref) / ref).mean().item()
    assert abs(off) <= room, off
    # the loss has the same lse beside a float z of at most a few units
    exact = ref - z.gather(1, y[:, None])[:, 0]
    off = ((loss.double() - exact) / ref).mean().item()
    assert abs(off) <= 2 * room, off
