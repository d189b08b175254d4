"""Rows of more elements than the head's calls take, also where 32 bits of their number would do: refused, before any
device work."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("cols", [Z.ZERO_HEAD_MAX_DIM + 8, 2 ** 32 + 8])
def test_too_many_columns(cols):
    row = torch.empty(cols, device="cuda", dtype=BF)
    x = row.view(1, cols)
    one = torch.zeros(1, device="cuda")
    target = torch.zeros(1, device="cuda", dtype=torch.int64)
    # (2^25 + 1 scales at most; one byte an element out of the row's own memory)
    scales = torch.empty(1, -(-cols // Z.ZERO_QUANT_BLOCK), device="cuda")
    codes = row.view(torch.int8)[:cols].view(1, cols)
    for call in (lambda: Z.residual_norm(x, None, row, 1e-5), lambda: Z.residual_norm_quantized(x, x, row, 1e-5),
                 lambda: Z.residual_norm_backward(x, row, x, None, 1e-5), lambda: Z.linear_loss(x, x, target),
                 lambda: Z.linear_loss_backward(x, x, target, one, one, grad_hidden=x, grad_weight=x),
                 lambda: Z.dequantize_rows(codes, scales, Z.ZERO_QUANT_INT8, BF)):
        with pytest.raises(Z.ZeroError, match="columns") as e:
            call()
        assert e.value.code == Z.ZERO_EINVAL
