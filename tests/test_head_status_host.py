"""The status word of the loss calls on the host (CPU only): threads that call first at once share one."""
import threading
import time

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z
from zero_partitioned_mixed_flat_gb300 import head


def test_threads_that_call_first_share_the_word(monkeypatch):
    zeros, waited = torch.zeros, []

    def slow(n, dtype, device):
        time.sleep(0.05)                                 # another thread gets here too
        return zeros(n, dtype=dtype)

    monkeypatch.setattr(head, "_STATUS", {})
    monkeypatch.setattr(head.torch, "zeros", slow)
    monkeypatch.setattr(head.torch.cuda, "synchronize", lambda device: waited.append(len(head._STATUS)))
    device, words = torch.device("cuda", 0), []
    threads = [threading.Thread(target=lambda: words.append(head._status(device))) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert len(words) == 8 and all(w is words[0] for w in words)
    assert waited == [0]                                 # nobody had it before the wait
    assert head._status(torch.device("cuda", 1)) is not words[0]


@pytest.mark.parametrize("code,status,bits", [(Z.ZERO_EINVAL, None, 4096), (Z.ZERO_EINVAL, 4096, None),
                                              (Z.ZERO_EALIGN, 4098, 4096), (Z.ZERO_EALIGN, 4096, 4097)])
def test_take_status_refuses(code, status, bits):
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_loss_take_status(status, bits, stream=0)
    assert e.value.code == code and Z.zero_last_error()
