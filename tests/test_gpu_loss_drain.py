"""Loss calls whose waits run out at different points: they end, say so, and leave nothing behind."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,d,v", [(300, 768, 2000), (700, 4096, 9000), (5, 72, 300)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_waits_that_run_out_anywhere(t, d, v, dtype):
    """Limits from nothing to more than a call takes: a call either reports the timeout or is right."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    h = torch.randn(t, d, generator=gen, device="cuda").to(dtype)
    w = (0.05 * torch.randn(v, d, generator=gen, device="cuda")).to(dtype)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    up = torch.rand(t, generator=gen, device="cuda")
    loss, lse = Z.linear_loss(h, w, y)
    grads = Z.linear_loss_backward(h, w, y, lse, up)
    Z.check_losses()
    gave_up = 0
    try:
        for limit in [0, 0, 100, 300, 700, 1000, 1500, 2000, 3000, 5000, 10000, 30000, 1000000]:
            Z.zero_loss_set_wait_limit(limit)
            for call, right in ((lambda: Z.linear_loss(h, w, y), (loss, lse)),
                                (lambda: Z.linear_loss_backward(h, w, y, lse, up), grads)):
                got = call()
                try:
                    Z.check_losses()
                except Z.ZeroError as e:
                    assert e.code == Z.ZERO_ETIMEOUT
                    gave_up += 1
                else:
                    assert all(torch.equal(a, b) for a, b in zip(got, right))
    finally:
        Z.zero_loss_set_wait_limit(4_000_000_000)
    assert gave_up >= 2                                  # the limits of 0
    got = Z.linear_loss(h, w, y) + Z.linear_loss_backward(h, w, y, lse, up)
    Z.check_losses()
    assert all(torch.equal(a, b) for a, b in zip(got, (loss, lse) + grads))
