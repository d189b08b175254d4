"""How far the forward pass's logits are off, beside data for which a sum loses nothing."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("t,d,v", [(300, 512, 400), (300, 1024, 400), (40, 4096, 300), (700, 4096, 30000), (9, 8200, 257)])
@pytest.mark.parametrize("few", [True, False])
def test_logits_whose_sums_are_exact(t, d, v, dtype, few):
    """Sums that no step rounds: one nonzero product (few), or small whole numbers throughout.

    Every logit is then the exact number.  What is left is the log-sum-exp's own: 4e-6 for its exponentials, their
    sum and its logarithm, and the rounding of lse and loss, 2^-23 of them.
    """
    gen = torch.Generator(device="cuda").manual_seed(t + d)
    w = torch.randint(-2, 3, (v, d), generator=gen, device="cuda").to(dtype)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    if few:
        h = torch.zeros(t, d, device="cuda")
        h[torch.arange(t), torch.randint(0, d, (t,), generator=gen, device="cuda")] = 15.0
        h = h.to(dtype)
    else:
        keep = torch.rand(t, d, generator=gen, device="cuda") < 40.0 / d
        h = torch.where(keep, torch.randint(-2, 3, (t, d), generator=gen, device="cuda"), 0).to(dtype)
    loss, lse = Z.linear_loss(h, w, y)
    z = h.double() @ w.double().t()
    ref = torch.logsumexp(z, 1)
    assert ((lse.double() - ref).abs() <= 4e-6 + ref.abs() * 2.0 ** -23).all()
    exact = ref - z.gather(1, y[:, None])[:, 0]
    assert ((loss.double() - exact).abs() <= 4e-6 + (ref.abs() + exact.abs()) * 2.0 ** -23).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [1024, 4096, 8200])
@pytest.mark.parametrize("t,v", [(200, 300), (700, 40000)])
def test_logits_that_are_all_of_lse(t, d, v, dtype):
    """One logit of 18 to 30, a sum that grows evenly over d products, and lse beside it.

    The tensor core drops what lies below the last place of its float sum at every step of 16 products: less than
    2^-23 of what the sum then is, and in fp16, whose products are longer, as much again as it aligns them.  A sum
    taken off after at most 512 products has at most 32 steps, on average half as large as at its end: 16.5 units of
    2^-23, of 2^-22 in fp16.  Beside that the parts' additions and the rounding of lse: a few 2^-24, taken as 4, and
    the 4e-6 of the exponentials over at least 18.  (Of 4096 products in one sum the mean would be 5.5e-6 in bf16.)
    """
    gen = torch.Generator(device="cuda").manual_seed(d)
    w = (torch.randn(v, d, generator=gen, device="cuda") * 0.02).to(dtype)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    high = 18 + 12 * torch.rand(t, 1, generator=gen, device="cuda")
    h = (0.1 * torch.randn(t, d, generator=gen, device="cuda") + high * w[y].float() / (0.0004 * d)).to(dtype)
    _, lse = Z.linear_loss(h, w, y)
    ref = torch.logsumexp(h.double() @ w.double().t(), 1)
    off = ((lse.double() - ref) / ref).mean().item()
    assert abs(off) <= 16.5 * 2.0 ** (-23 if dtype == BF else -22) + 4 * 2.0 ** -24 + 4e-6 / 18, off
