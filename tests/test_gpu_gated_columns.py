"""Rows of more elements than the gated projections take, also where 32 bits of their number would do: refused, before
any device work."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [Z.ZERO_HEAD_MAX_DIM + 8, 2 ** 32 + 8])
def test_too_many_columns(cols):
    space = torch.empty(cols + 7 * 64, device="cuda", dtype=torch.bfloat16)      # rows that overlap: no more memory
    x, gate, up = space[:cols].view(1, cols), space.as_strided((8, cols), (64, 1)), space.as_strided((8, cols), (64, 1))
    grad = torch.zeros(1, 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(Z.ZeroError, match="columns") as e:
        Z.gated_linear(x, gate, up)
    assert e.value.code == Z.ZERO_EINVAL
    with pytest.raises(Z.ZeroError, match="columns") as e:
        Z.gated_linear_backward(x, gate, up, grad, grad_x=x, grad_gate=gate, grad_up=up)
    assert e.value.code == Z.ZERO_EINVAL
