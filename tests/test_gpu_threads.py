"""A thread whose first CUDA call is one of the library's: every buffer is there already, so nothing has bound the
device's context to the thread before."""
import threading

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def in_a_new_thread(call):
    raised = []

    def work():
        try:
            call()
        except Exception as e:   # noqa: BLE001  (reported below)
            raised.append(e)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join(120)
    assert not thread.is_alive() and not raised, raised
    torch.cuda.synchronize()


def rows(t, d, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(t + d)
    return (torch.randn(t, d, generator=gen, device="cuda") * std).to(BF)


@pytest.mark.parametrize("t", [3, 60, 300])
def test_gated_projections(t):
    x, gate, up, grad = rows(t, 264), rows(520, 264, 0.1), rows(520, 264, 0.1).flip(0).contiguous(), rows(t, 520)
    want = (Z.gated_linear(x, gate, up), *Z.gated_linear_backward(x, gate, up, grad))
    out, gx, gg, gu = (torch.empty_like(w) for w in want)
    need = Z.zero_gated_workspace(t, 520, 264)[1]
    space, status = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    shape = (x, 264, gate, 264, up, 264, Z.ZERO_ACT_SILU)
    in_a_new_thread(lambda: Z.zero_gated_forward(*shape, t, 520, 264, Z.ZERO_BF16, out, 520, status, None, 0, stream=0))
    in_a_new_thread(lambda: Z.zero_gated_backward(*shape, grad, 520, t, 520, 264, Z.ZERO_BF16, gx, 264, gg, 264, gu, 264, status,
                                                  space, need, stream=0))
    assert all(torch.equal(a, b) for a, b in zip((out, gx, gg, gu), want)) and int(status) == 0


@pytest.mark.parametrize("t", [3, 300])
def test_loss(t):
    h, w = rows(t, 264), rows(5000, 264)
    y = torch.arange(t, device="cuda")
    up = torch.ones(t, device="cuda")
    want_loss, want_lse = Z.linear_loss(h, w, y)
    want_h, want_w = Z.linear_loss_backward(h, w, y, want_lse, up)
    loss, lse, gh, gw = (torch.empty_like(x) for x in (want_loss, want_lse, want_h, want_w))
    forward, backward = Z.zero_loss_workspace(t, 5000, 264)
    space, status = torch.empty(max(forward, backward), dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    shape = (h, 264, w, 264, y, -100, t, 5000, 264, Z.ZERO_BF16)
    in_a_new_thread(lambda: Z.zero_loss_forward(*shape, loss, lse, status, space, forward, stream=0))
    in_a_new_thread(lambda: Z.zero_loss_backward(*shape, lse, up, gh, 264, gw, 264, status, space, backward, stream=0))
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, gh, gw), (want_loss, want_lse, want_h, want_w))) and int(status) == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw(bits):
    def case():
        p = [torch.linspace(-1, 1, 3000, device="cuda")]
        return p, [torch.linspace(1, 2, 3000, device="cuda")], Z.adamw_state(p, bits)
    a, b = case(), case()
    Z.adamw_step(*a, 1e-2)
    in_a_new_thread(lambda: Z.adamw_step(*b, 1e-2, stream=0))
    assert torch.equal(a[0][0], b[0][0]) and torch.equal(a[2].m, b[2].m) and int(b[2].record[0]) == 1
