"""The word that the loss calls report through: nothing that a call sets is lost, whoever else calls."""
import threading

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu


def batch(t=40, d=64, v=100, key=0):
    gen = torch.Generator(device="cuda").manual_seed(key)
    h = torch.randn(t, d, generator=gen, device="cuda").bfloat16()
    w = torch.randn(v, d, generator=gen, device="cuda").bfloat16()
    return h, w, torch.randint(0, v, (t,), generator=gen, device="cuda")


def test_a_bit_set_while_another_check_ends_is_kept(monkeypatch):
    """A call that meets a bad target just after another thread's check has read the word."""
    h, w, y = batch()
    bad = y.clone()
    bad[3] = 1000
    Z.check_losses()
    read = torch.Tensor.item
    late = []

    def item(tensor):
        value = read(tensor)
        if not late:
            late.append(True)
            Z.linear_loss(h, w, bad)
            torch.cuda.synchronize()
        return value

    monkeypatch.setattr(torch.Tensor, "item", item)
    Z.check_losses()
    monkeypatch.undo()
    assert late
    with pytest.raises(Z.ZeroError) as e:
        Z.check_losses()
    assert e.value.code == Z.ZERO_EINVAL
    Z.check_losses()


def test_losses_on_streams_at_once():
    """Calls of four threads, each on a stream of its own and none waiting for another, equal calls alone."""
    cases = [batch(t, d, v, t) for t, d, v in ((3, 768, 9000), (300, 768, 9000), (700, 264, 5000), (40, 1600, 20000))]
    ups = [torch.rand(len(y), device="cuda") for _, _, y in cases]
    alone = []
    for (h, w, y), up in zip(cases, ups):
        loss, lse = Z.linear_loss(h, w, y)
        alone.append((loss, lse) + Z.linear_loss_backward(h, w, y, lse, up))
    torch.cuda.synchronize()
    streams, wrong = [torch.cuda.Stream() for _ in cases], []
    start = threading.Barrier(len(cases))

    def work(i):
        (h, w, y), up = cases[i], ups[i]
        start.wait()
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                loss, lse = Z.linear_loss(h, w, y)
                got = (loss, lse) + Z.linear_loss_backward(h, w, y, lse, up)
                wrong.append(sum((a != b).sum() for a, b in zip(got, alone[i])))
        streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for thread in threads:
        thread.start()
    for thread in threads:
        thread.join(120)
    assert not any(thread.is_alive() for thread in threads)
    assert len(wrong) == 20 * len(cases) and sum(int(n) for n in wrong) == 0
    Z.check_losses()
