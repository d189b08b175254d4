"""The norm at the ends of its types' ranges: rows with NaN and infinities in its 8-bit form, rows whose squares leave float's range."""
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


# ---- rows whose squares leave float's range -----------------------------------------------

# float error of the sum, of rstd (a subnormal float above 2^126: 2^-22 of itself) and of the products
NORM_FLOAT = 40 * 2.0 ** -24


def close(got, ref, extra):
    """bfloat16 of a value whose float error is `extra`: half of 2^-7 of itself, or of the least step."""
    room = ref.abs() * (2.0 ** -8 * 1.001) + 2.0 ** -134 + extra
    assert not (got.isnan() | ref.isnan()).any()
    worst = ((got.double() - ref).abs() / room).max().item()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("rows,dim", [(3, 64), (160, 1024), (200, 1600), (40, 4104), (170, 16384)])
@pytest.mark.parametrize("size,eps", [(1e19, EPS), (4e19, 0.0), (1e30, EPS), (3e37, EPS), (1e-20, 0.0), (1e-25, 0.0), (1e-36, 0.0),
                                      (1e-25, 1e-38)])
def test_norm_of_rows_whose_squares_leave_floats_range(rows, dim, size, eps):
    """Finite rows have a finite norm, and its gradients, however large or small they are."""
    x, r = rows_of(dim, rows, dim, BF, size), rows_of(dim + 1, rows, dim, BF, size)
    x[1], r[1] = rows_of(7, 2, dim, BF).unbind()         # an ordinary row between them
    w = (1 + 0.1 * rows_of(dim + 2, 1, dim, BF)[0].float()).to(BF)
    out, total = Z.residual_norm(x, r, w, eps)
    s = x.double() + r.double()
    rstd = (s.square().mean(1, keepdim=True) + eps).rsqrt()
    ref = s * rstd * w.double()
    close(out, ref, ref.abs() * NORM_FLOAT)
    close(total, s, s.abs() * 2.0 ** -23)
    codes, scales, _ = Z.residual_norm_quantized(x, r, w, eps, Z.ZERO_QUANT_INT8)
    top = blocks_of(ref.abs()).amax(2)
    assert ((scales.double() - top / 127).abs() <= top / 127 * (NORM_FLOAT + 2.0 ** -24)).all()
    wide = scales.double().repeat_interleave(128, 1)[:, :dim]
    assert ((codes.double() * wide - ref).abs() <= wide * 0.5 * (1 + 1e-6) + ref.abs() * 2 * NORM_FLOAT).all()
    S, W = total.double(), w.double()
    gy = rows_of(dim + 3, rows, dim, BF, 0.3)
    G = gy.double()
    gs = rows_of(dim + 4, rows, dim, BF, 0.3)
    rstd = (S.square().mean(1, keepdim=True) + eps).rsqrt()
    unit = S * rstd
    for extra in (gs, None):
        gi, gw = Z.residual_norm_backward(total, w, gy, extra, eps)
        more = 0.0 if extra is None else extra.double()
        ref = rstd * (W * G - unit * (W * G * unit).mean(1, keepdim=True)) + more
        spread = (W * G * unit).abs().mean(1, keepdim=True) * rstd * unit.abs()
        terms = rstd * (W * G).abs() + spread + (0.0 if extra is None else more.abs())
        close(gi, ref, NORM_FLOAT * (terms + 2 * spread))
        per = G * unit
        close(gw, per.sum(0), (rows + 64) * 2.0 ** -24 * per.abs().sum(0))


def test_norm_of_one_large_element():
    """An element whose square alone leaves float's range: the others' share is what is left of them."""
    x = rows_of(1, 200, 768, BF)
    x[:, 5] = 3e38
    x[7] = 0.0
    x[8] = torch.where(x[8] < 0, -3e38, 3e38)            # rstd is a subnormal float
    w = torch.ones(768, dtype=BF, device="cuda")
    out, _ = Z.residual_norm(x, None, w, EPS)
    s = x.double()
    ref = s * (s.square().mean(1, keepdim=True) + EPS).rsqrt()
    close(out, ref, ref.abs() * NORM_FLOAT)
    assert (out[7] == 0).all()
