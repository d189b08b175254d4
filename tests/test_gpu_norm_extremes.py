"""The norm at the ends of its types' ranges: rows with NaN and infinities in its 8-bit form."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
EPS = 1e-5
NAN, INF = float("nan"), float("inf")


def rows_of(key, rows, dim, dtype, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(key)
    return (torch.randn(rows, dim, generator=gen, device="cuda") * std).to(dtype)


def blocks_of(values):
    """[rows, blocks, 128], the last block of a row filled up with zeros."""
    return torch.nn.functional.pad(values, (0, -values.shape[1] % 128)).unflatten(1, (-1, 128))


@pytest.mark.parametrize("fmt", [Z.ZERO_QUANT_INT8, Z.ZERO_QUANT_FP8_E4M3])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows,dim", [(7, 24), (300, 264), (300, 1032), (160, 8200), (7, 16384)])
def test_quantized_norm_keeps_what_is_not_finite(rows, dim, dtype, fmt):
    """A NaN or an infinity comes back as NaN wherever the 16-bit form has NaN, and no other row knows of it."""
    x, r = rows_of(dim, rows, dim, dtype), rows_of(dim + 1, rows, dim, dtype)
    w = rows_of(dim + 2, 1, dim, dtype)[0].contiguous()
    clean = Z.residual_norm_quantized(x, r, w, EPS, fmt)
    x[1, 3], x[3, dim - 1], r[4, dim // 2], r[5, 0] = NAN, INF, -INF, NAN
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[1, 3, 4, 5]] = True
    codes, scales, total = Z.residual_norm_quantized(x, r, w, EPS, fmt)
    out, total16 = Z.residual_norm(x, r, w, EPS)
    back = Z.dequantize_rows(codes, scales, fmt, dtype)
    for got, was in ((codes, clean[0]), (scales, clean[1]), (total, clean[2])):
        assert torch.equal(got[~bad], was[~bad])
    assert torch.equal(total.isnan(), total16.isnan()) and total[3, dim - 1].isinf()
    lost = blocks_of(out.isnan().float()).amax(2) > 0        # blocks with a NaN
    assert lost[bad].any(1).all() and not lost[~bad].any()
    assert torch.equal(scales.isnan(), lost)
    assert torch.equal(blocks_of(back.isnan().float()).amax(2) > 0, lost)
    assert back[out.isnan()].isnan().all() and back[~out.isnan() & ~back.isnan()].isfinite().all()


@pytest.mark.parametrize("fmt", [Z.ZERO_QUANT_INT8, Z.ZERO_QUANT_FP8_E4M3])
def test_quantized_norm_of_a_weight_that_is_not_finite(fmt):
    """A NaN in the weight costs its own block of every row, not the others."""
    x, w = rows_of(3, 20, 520, BF), rows_of(4, 1, 520, BF)[0].contiguous()
    clean = Z.residual_norm_quantized(x, None, w, EPS, fmt)
    w[200] = NAN
    codes, scales, _ = Z.residual_norm_quantized(x, None, w, EPS, fmt)
    assert scales[:, 1].isnan().all()
    rest = [0, 2, 3, 4]
    assert torch.equal(scales[:, rest], clean[1][:, rest])
    assert torch.equal(codes[:, :128], clean[0][:, :128]) and torch.equal(codes[:, 256:], clean[0][:, 256:])
    assert Z.dequantize_rows(codes, scales, fmt, BF)[:, 128:256].isnan().all()
