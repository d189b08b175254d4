"""train_head's options on the host: what cannot go together is refused before any device work."""
import sys

import pytest

from zero_partitioned_mixed_flat_gb300 import train_head


@pytest.mark.parametrize("moments", ["8", "32"])
def test_moments_and_ranks_do_not_go_together(moments, monkeypatch, capsys):
    monkeypatch.setattr(train_head, "train_whole", lambda *a, **k: [0.0])
    monkeypatch.setattr(sys, "argv", ["train_head", "--moments", moments, "--ranks", "2"])
    with pytest.raises(SystemExit) as e:
        train_head.main()
    assert e.value.code == 2 and "--ranks" in capsys.readouterr().err


@pytest.mark.parametrize("more,ranks", [([], 2), (["--ranks", "3"], 3)])
def test_ranks_of_the_partitioned_step(more, ranks, monkeypatch):
    seen = []
    monkeypatch.setattr(train_head, "train", lambda steps, n, wide: seen.append((steps, n, wide)) or [0.0])
    monkeypatch.setattr(sys, "argv", ["train_head", "--steps", "5", *more])
    train_head.main()
    assert seen == [(5, ranks, 0)]
