"""The training head on the GPU against plain implementations in 64 bits.

Tolerances are derived, not fitted.  u is half a unit in the last place of the
16-bit type (2^-8 bfloat16, 2^-11 float16, relative), `least` half its smallest step.  A
value that is computed in float and rounded once to 16 bits is within
u |ref| + least of the exact value, plus the float arithmetic's own error, for
which each test states a bound on the terms that enter the sum.
"""
import math

import numpy as np
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
EPS = 1e-5


def half_ulp(dtype):
    return (2.0 ** -8, 2.0 ** -134) if dtype == BF else (2.0 ** -11, 2.0 ** -25)


def close(got, ref, dtype, extra=0.0):
    """|got - ref| <= u |ref| + least + extra (a tensor or a number), element by element."""
    u, least = half_ulp(dtype)
    got, room = got.double(), ref.abs() * (u * 1.001) + least + extra
    worst = ((got - ref).abs() / room).max().item() if ref.numel() else 0.0
    assert not (got.isnan() | ref.isnan()).any()
    assert worst <= 1.0, worst


def rows_of(gen, rows, dim, dtype, std=1.0, pad=0):
    return (torch.randn(rows, dim + pad, generator=gen, device="cuda") * std).to(dtype)[:, :dim]


def seeded(*key):
    g = torch.Generator(device="cuda")
    g.manual_seed(hash(key) % (2 ** 31))
    return g


# ---- residual addition + RMS norm --------------------------------------------------

def norm64(x, residual, weight, eps=EPS):
    s = x.double() + (0.0 if residual is None else residual.double())
    rstd = (s.square().mean(1, keepdim=True) + eps).rsqrt()
    return s * rstd * weight.double(), s, rstd


# float error of s, of the mean of squares (a tree over at most 16384 / 16 leaves of a
# thread's 32: under 64 roundings), of rsqrt and of two products
NORM_FLOAT = 40 * 2.0 ** -24

SHAPES = [(1, 8), (3, 64), (1, 16384), (2, 72), (151, 264), (152, 1024), (153, 1032), (1000, 1600), (300, 2056),
          (17, 4096), (400, 4104), (200, 8200), (160, 16384), (1023, 768)]


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_forward(rows, dim, dtype):
    gen = seeded(rows, dim)
    pad = 8 * (rows % 3)
    x, r = rows_of(gen, rows, dim, dtype, 0.5, pad), rows_of(gen, rows, dim, dtype, 2.0, pad)
    w = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(dtype)
    for residual in (r, None):
        out, total = Z.residual_norm(x, residual, w, EPS)
        ref, s, _ = norm64(x, residual, w)
        close(out, ref, dtype, ref.abs() * NORM_FLOAT)
        close(total, s, dtype, s.abs() * 2.0 ** -23)


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("fmt", [Z.ZERO_QUANT_INT8, Z.ZERO_QUANT_FP8_E4M3])
def test_norm_quantized(rows, dim, dtype, fmt):
    gen = seeded(rows, dim, fmt)
    x, r = rows_of(gen, rows, dim, dtype, 0.5, 8), rows_of(gen, rows, dim, dtype, 2.0)
    x[0] = 0
    r[0] = 0                                            # a row of zeros
    if dim > 128:
        x[-1, :128] = 0
        r[-1, :128] = 0                                 # a block of zeros
    w = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(dtype)
    codes, scales, total = Z.residual_norm_quantized(x, r, w, EPS, fmt)
    ref, s, _ = norm64(x, r, w)
    close(total, s, dtype, s.abs() * 2.0 ** -23)
    blocks = -(-dim // 128)
    padded = torch.nn.functional.pad(ref, (0, blocks * 128 - dim)).view(rows, blocks, 128)
    top = padded.abs().amax(2)
    wide = scales.double().repeat_interleave(128, 1)[:, :dim]
    assert scales.shape == (rows, blocks)
    assert (scales[0] == 0).all() and (codes[0] == 0).all()
    if fmt == Z.ZERO_QUANT_INT8:
        assert ((scales.double() - top / 127).abs() <= top / 127 * (NORM_FLOAT + 2.0 ** -24)).all()
        assert codes.min() >= -127
        # half a step, and the value's own float error
        assert ((codes.double() * wide - ref).abs() <= wide * 0.5 * (1 + 1e-6) + ref.abs() * 2 * NORM_FLOAT).all()
    else:
        # a power of two that puts the largest magnitude into [128, 256)
        assert (scales[top > 0].log2() == scales[top > 0].log2().round()).all()
        lead = top[top > 0] / scales.double()[top > 0]
        assert ((lead >= 128 * (1 - NORM_FLOAT)) & (lead < 256 * (1 + NORM_FLOAT))).all()
        value = codes.view(torch.float8_e4m3fn).double() * wide
        # E4M3: half of 2^-3 of the leading power of two, at least half of 2^-9
        assert ((value - ref).abs() <= torch.maximum(ref.abs() * 2.0 ** -4, wide * 2.0 ** -10) * (1 + 1e-6)).all()
    back = Z.dequantize_rows(codes, scales, fmt, dtype)
    value = codes.double() if fmt == Z.ZERO_QUANT_INT8 else codes.view(torch.float8_e4m3fn).double()
    close(back, value * wide, dtype, (value * wide).abs() * 2.0 ** -23)


def test_quantized_norm_is_the_shard_quantizer():
    """Where the norm's values are 16-bit numbers, its codes are those of zero_quantize_shard, bit for bit."""
    rows, dim = 64, 1024
    gen = seeded(7)
    # rows whose mean square is exactly 1, weight and result powers of two
    x = torch.where(torch.rand(rows, dim, generator=gen, device="cuda") < 0.5, 1.0, -1.0).to(BF)
    w = torch.randn(dim, generator=gen, device="cuda").to(BF)
    plan = Z.ZeroPlan(rows * dim, 1, None, 128, 3, None, Z.ZERO_BF16)
    for fmt in (Z.ZERO_QUANT_INT8, Z.ZERO_QUANT_FP8_E4M3):
        codes, scales, _ = Z.residual_norm_quantized(x, None, w, 0.0, fmt)
        plan.set_gather_quantization(fmt)
        shard = (x.float() * w.float()).to(BF).reshape(-1)
        c2 = torch.empty(rows * dim, dtype=torch.int8, device="cuda")
        s2 = torch.empty(rows * dim // 128, device="cuda")
        plan.quantize(shard, c2, s2)
        assert torch.equal(codes.reshape(-1), c2) and torch.equal(scales.reshape(-1), s2)
    plan.close()


def test_dequantize_every_code():
    codes = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).view(torch.int8).repeat(3, 1)
    scales = torch.tensor([[1.0, 0.25], [3.0, 2.0 ** -20], [0.0, 7.0]], device="cuda")
    wide = scales.repeat_interleave(128, 1)
    for dtype in (BF, FP):
        got = Z.dequantize_rows(codes, scales, Z.ZERO_QUANT_INT8, dtype)
        assert torch.equal(got, (codes.float() * wide).to(dtype))
        got = Z.dequantize_rows(codes, scales, Z.ZERO_QUANT_FP8_E4M3, dtype)
        ref = (codes.view(torch.float8_e4m3fn).float() * wide).to(dtype)
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got[~ref.isnan()], ref[~ref.isnan()])


def test_norm_in_place_streams_and_empty():
    gen = seeded(11)
    x, r, w = rows_of(gen, 500, 1600, BF), rows_of(gen, 500, 1600, BF), rows_of(gen, 1, 1600, BF)[0].contiguous()
    out, total = Z.residual_norm(x, r, w, EPS)
    out2, total2 = Z.residual_norm(x, r, w, EPS)
    assert torch.equal(out, out2) and torch.equal(total, total2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out3, total3 = Z.residual_norm(x, r, w, EPS, stream=side)
    out4, _ = Z.residual_norm(x, r, w, EPS, stream=int(side.cuda_stream))
    side.synchronize()
    assert torch.equal(out, out3) and torch.equal(total, total3) and torch.equal(out, out4)
    # the sum in the residual's place, as a residual stream is kept
    keep, same = r.clone(), torch.empty_like(out)
    Z.zero_norm_forward(x, 1600, keep, 1600, w, EPS, 500, 1600, Z.ZERO_BF16, same, 1600, keep, 1600)
    assert torch.equal(keep, total) and torch.equal(same, out)
    # no sum asked for
    Z.zero_norm_forward(x, 1600, r, 1600, w, EPS, 500, 1600, Z.ZERO_BF16, same, 1600, None, 0)
    assert torch.equal(same, out)
    for n in (0,):
        a, b = Z.residual_norm(x[:n], r[:n], w, EPS)
        assert a.shape == (0, 1600) and b.shape == (0, 1600)
        gi, gw = Z.residual_norm_backward(b, w, a, None, EPS)
        assert gi.shape == (0, 1600) and (gw == 0).all()
        c, s, _ = Z.residual_norm_quantized(x[:n], None, w, EPS)
        assert Z.dequantize_rows(c, s, 0, BF).shape == (0, 1600)


def test_norm_rows_do_not_touch_each_other():
    """A row with an infinity or a NaN leaves the others as they are."""
    gen = seeded(12)
    x, w = rows_of(gen, 300, 1032, FP), rows_of(gen, 1, 1032, FP)[0].contiguous()
    g = rows_of(gen, 300, 1032, FP)
    out, _ = Z.residual_norm(x, None, w, EPS)
    gi, _ = Z.residual_norm_backward(x, w, g, None, EPS)
    y = x.clone()
    y[5, 3], y[77, 1031], y[299] = float("inf"), float("nan"), 0.0
    out2, total2 = Z.residual_norm(y, None, w, EPS)
    gi2, _ = Z.residual_norm_backward(y, w, g, None, EPS)
    rest = torch.ones(300, dtype=torch.bool, device="cuda")
    rest[[5, 77, 299]] = False
    assert torch.equal(out[rest], out2[rest]) and torch.equal(gi[rest], gi2[rest])
    assert out2[77].isnan().all() and out2[5, 3].isnan() and (out2[299] == 0).all() and total2[5, 3].isinf()


def test_norm_keeps_the_sign_of_zero():
    x = torch.zeros(2, 64, dtype=BF, device="cuda")
    x[0] = -0.0
    _, total = Z.residual_norm(x, None, torch.ones(64, dtype=BF, device="cuda"), EPS)
    assert torch.equal(total.view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("rows,dim", SHAPES + [(5000, 768), (2500, 1600), (3000, 24)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_backward(rows, dim, dtype):
    gen = seeded(rows, dim, 1)
    s = rows_of(gen, rows, dim, dtype, 2.0, 8 * (dim % 3))
    w = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(dtype)
    gy, gs = rows_of(gen, rows, dim, dtype, 0.3, 16), rows_of(gen, rows, dim, dtype, 0.3)
    for extra in (gs, None):
        gi, gw = Z.residual_norm_backward(s, w, gy, extra, EPS)
        S, W, G = s.double(), w.double(), gy.double()
        rstd = (S.square().mean(1, keepdim=True) + EPS).rsqrt()
        along = (W * G * S).mean(1, keepdim=True) * rstd.square()
        ref = rstd * (W * G - S * along) + (0.0 if extra is None else extra.double())
        # the mean's terms cancel: its float error is relative to the sum of their magnitudes
        spread = (W * G * S).abs().mean(1, keepdim=True) * rstd.square() * rstd * S.abs()
        terms = rstd * ((W * G).abs() + (S * along).abs()) + (0.0 if extra is None else extra.double().abs())
        close(gi, ref, dtype, NORM_FLOAT * (terms + 2 * spread))
        per = G * S * rstd
        close(gw, per.sum(0), dtype, (rows + 64) * 2.0 ** -24 * per.abs().sum(0))
        again = Z.residual_norm_backward(s, w, gy, extra, EPS)
        assert torch.equal(again[0], gi) and torch.equal(again[1], gw)


def test_norm_backward_against_differences():
    """The gradients against central differences of the 64-bit forward."""
    rows, dim = 6, 72
    gen = seeded(31)
    s, w, gy = rows_of(gen, rows, dim, FP), rows_of(gen, 1, dim, FP)[0].contiguous(), rows_of(gen, rows, dim, FP)
    gi, gw = Z.residual_norm_backward(s, w, gy, None, EPS)

    def value(S, W):
        return ((S * (S.square().mean(1, keepdim=True) + EPS).rsqrt() * W) * gy.double()).sum().item()

    S, W, step = s.double(), w.double(), 1e-5
    u, least = half_ulp(FP)
    for k in range(40):
        i, j = (k * 7) % rows, (k * 31) % dim
        d = torch.zeros_like(S)
        d[i, j] = step
        slope = (value(S + d, W) - value(S - d, W)) / (2 * step)
        # step^2 of the third derivative (order 1), and 1e-16 / step of the difference
        assert abs(gi[i, j].item() - slope) <= u * abs(slope) * 1.01 + least + 1e-5
        e = torch.zeros_like(W)
        e[j] = step
        slope = (value(S, W + e) - value(S, W - e)) / (2 * step)
        assert abs(gw[j].item() - slope) <= u * abs(slope) * 1.01 + least + 1e-5


def test_norm_offsets_beyond_32_bits():
    """Rows whose byte and element offsets pass 2^32 and 2^31."""
    rows, dim = 140000, 16384
    x = torch.zeros(rows, dim, dtype=BF, device="cuda")
    gen = seeded(99)
    x[-3:] = rows_of(gen, 3, dim, BF)
    w = rows_of(gen, 1, dim, BF)[0].contiguous()
    out, total = Z.residual_norm(x, None, w, EPS)
    ref, s, _ = norm64(x[-3:], None, w)
    close(out[-3:], ref, BF, ref.abs() * NORM_FLOAT)
    assert torch.equal(total[-3:], x[-3:]) and (out[:-3] == 0).all()
    del out
    codes, scales, _ = Z.residual_norm_quantized(x, None, w, EPS, Z.ZERO_QUANT_INT8)
    del _
    back = Z.dequantize_rows(codes, scales, Z.ZERO_QUANT_INT8, BF)
    step = scales[-3:].double().repeat_interleave(128, 1)
    close(back[-3:], ref, BF, step * 0.5 * (1 + 1e-6) + ref.abs() * 2 * NORM_FLOAT)
    assert (back[:-3] == 0).all()
    del back, codes
    g = torch.zeros(rows, dim, dtype=BF, device="cuda")
    g[-3:] = rows_of(gen, 3, dim, BF)
    gi, gw = Z.residual_norm_backward(total, w, g, None, EPS)
    S, W, G = x[-3:].double(), w.double(), g[-3:].double()
    rstd = (S.square().mean(1, keepdim=True) + EPS).rsqrt()
    per = G * S * rstd
    close(gw, per.sum(0), BF, 64 * 2.0 ** -24 * per.abs().sum(0))
    small, _ = Z.residual_norm_backward(x[-3:].contiguous(), w, g[-3:].contiguous(), None, EPS)
    # the same row by another number of threads: both within the bound of the exact value
    along = (W * G * S).mean(1, keepdim=True) * rstd.square()
    ref = rstd * (W * G - S * along)
    spread = (W * G * S).abs().mean(1, keepdim=True) * rstd.square() * rstd * S.abs()
    terms = rstd * ((W * G).abs() + (S * along).abs())
    for got in (gi[-3:], small):
        close(got, ref, BF, NORM_FLOAT * (terms + 2 * spread))


# ---- cross entropy -------------------------------------------------------------------

def loss64(h, w, y, ignore=-100):
    z = h.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    counts = (y != ignore) & (y >= 0) & (y < w.shape[0])
    at = torch.where(counts, y, 0)
    loss = torch.where(counts, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    return z, lse, loss, counts, at


def logit_error(h, w):
    """Bound on a logit's float error: each of a sum's at most 32 steps of 16 products, and
    each of the additions of such sums, loses at most 2^-22 of the magnitudes added."""
    most = (h.double().abs() @ w.double().abs().t()).amax()
    return (34 + h.shape[1] / 512) * 2.0 ** -22 * most.item()


def check_loss(h, w, y, grad_loss, ignore=-100, seeded_lse=None):
    dtype = h.dtype
    loss, lse = Z.linear_loss(h, w, y, ignore=ignore)
    z, ref_lse, ref_loss, counts, at = loss64(h, w, y, ignore)
    ez = logit_error(h, w)
    # the sum of exponentials: 2e-6 for the exponential and its argument, and its additions
    e_lse = ez + 4e-6 + ref_lse.abs() * 2.0 ** -23
    assert ((lse.double() - ref_lse).abs() <= e_lse).all()
    assert ((loss.double() - ref_loss).abs() <= e_lse + ez + ref_loss.abs() * 2.0 ** -23).all()
    assert (loss[~counts & (y == ignore)] == 0).all()
    gh, gw = Z.linear_loss_backward(h, w, y, lse, grad_loss, ignore=ignore)
    q = torch.exp(z - ref_lse[:, None])
    q[torch.arange(len(y), device="cuda"), at] -= 1.0
    q *= torch.where(counts, grad_loss, 0.0).double()[:, None]
    # q is rounded to 16 bits: u of itself, its exponential's error, and in fp16 half a
    # step of 2^-24 on a scale where the largest |grad_loss| is 2^15; then float sums
    u, _ = half_ulp(dtype)
    top = torch.where(counts, grad_loss.abs(), 0.0).max().item() if len(y) else 0.0
    slack = 2 * ez + 1e-5
    p = torch.exp(z - ref_lse[:, None]) * torch.where(counts, grad_loss.abs(), 0.0).double()[:, None]
    eq = q.abs() * (u * 1.01) + p * slack + (top * 2.0 ** -40 if dtype == FP else 0.0)
    steps = 2.0 ** -22
    for got, ref, err in ((gh, q @ w.double(), (eq + q.abs() * (w.shape[0] / 16 + 64) * steps) @ w.double().abs()),
                          (gw, q.t() @ torch.where(counts[:, None], h.double(), 0.0),
                           (eq + q.abs() * (len(y) / 16 + 64) * steps).t() @ torch.where(counts[:, None], h.double().abs(), 0.0))):
        close(got, ref, dtype, err)
    assert (gh[~counts] == 0).all()
    Z.check_losses()
    return loss, lse, gh, gw


def case(t, d, v, dtype, ignored=0.0, pad=0, key=0):
    gen = seeded(t, d, v, key)
    h, w = rows_of(gen, t, d, dtype, 1.0, pad), rows_of(gen, v, d, dtype, 0.05, pad)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    y = torch.where(torch.rand(t, generator=gen, device="cuda") < ignored, -100, y)
    g = torch.rand(t, generator=gen, device="cuda") - 0.3
    return h, w, y, g


LOSSES = [(1, 8, 1), (1, 64, 257), (2, 72, 300), (3, 1600, 77), (4, 768, 5003), (5, 768, 5003), (1, 16384, 130),
          (4, 16384, 129), (127, 520, 255), (128, 64, 256), (129, 136, 257), (255, 200, 512), (256, 1032, 513),
          (257, 264, 1000), (300, 4096, 700), (700, 96, 20011), (1025, 776, 3000), (513, 8, 2049), (64, 16384, 520)]


@pytest.mark.parametrize("t,d,v", LOSSES)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_loss(t, d, v, dtype):
    check_loss(*case(t, d, v, dtype, pad=8 * (v % 3)))


@pytest.mark.parametrize("ignored", [0.05, 0.5, 0.97, 1.1])
@pytest.mark.parametrize("t,d,v", [(1, 64, 70), (3, 64, 300), (130, 136, 257), (600, 264, 1999), (1025, 72, 513)])
def test_loss_ignored_tokens(t, d, v, ignored):
    check_loss(*case(t, d, v, FP, ignored), )
    h, w, y, g = case(t, d, v, BF, ignored, 8)
    y2 = torch.where(y == -100, 7, y.clamp(max=6))      # another number means "ignore"
    y2 = torch.where((y2 != 7) & (y2 >= v), 0, y2)
    check_loss(h, w, y2, g, ignore=7)


@pytest.mark.parametrize("t", [4095, 4096, 4097, 5121, 9001])
@pytest.mark.parametrize("ignored", [0.3, 0.999, 0.0])
def test_loss_many_tokens_some_ignored(t, ignored):
    """The counted tokens are copied by the launch that finds them up to 4096 tokens, and by another beyond."""
    check_loss(*case(t, 72, 300, BF, ignored, 8))


@pytest.mark.parametrize("t,counted", [(1, 1), (2, 1), (3, 3), (7, 7), (31, 31), (32, 32), (33, 32), (40, 5), (63, 32), (64, 32),
                                       (65, 2), (300, 9), (4096, 32), (4097, 1), (5000, 30)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_loss_few_counted_tokens_round_gradients_once(t, counted, dtype):
    """One slope is most of such a gradient: its rounding to 16 bits must not be the gradient's error.

    The bound: the gradients' relative error (in norm) is that of rounding the exact ones once, e, but for the
    logits' error.  72 products are five steps of the tensor core, each at most 2^-22 off of sums of magnitudes
    up to about 2^6 here: 8e-5 at the worst and for all at once, a tenth of it in norm over entries whose errors
    differ.  So 1.05 e + 1e-5; with slopes rounded to 16 bits one token's error is about 1.4 e.
    """
    d, v = 72, 700
    total = torch.zeros(4, dtype=torch.float64)
    for key in range(8):
        gen = seeded(t, counted, key)
        w = rows_of(gen, v, d, dtype, 0.05)
        y = torch.randint(0, v, (t,), generator=gen, device="cuda")
        above = 8.0 * torch.rand(t, 1, generator=gen, device="cuda")   # targets that are likely, to a different extent
        h = (torch.randn(t, d, generator=gen, device="cuda") + above * w[y].float() / (0.05 ** 2 * d)).to(dtype)
        g = 0.5 + torch.rand(t, generator=gen, device="cuda")
        keep = torch.zeros(t, dtype=torch.bool, device="cuda")
        keep[torch.randperm(t, generator=gen, device="cuda")[:counted]] = True
        y = torch.where(keep, y, -100)
        z, lse64, _, counts, at = loss64(h, w, y)
        q = torch.exp(z - lse64[:, None])
        q[torch.arange(t, device="cuda"), at] -= 1.0
        q *= torch.where(counts, g, 0.0).double()[:, None]
        gh, gw = Z.linear_loss_backward(h, w, y, Z.linear_loss(h, w, y)[1], g)
        for i, (got, ref) in enumerate(((gh, q @ w.double()), (gw, q.t() @ h.double()))):
            total[2 * i] += ((got.double() - ref).norm() / ref.norm()).item() / 8
            total[2 * i + 1] += ((ref.to(dtype).double() - ref).norm() / ref.norm()).item() / 8
        assert (gh[~keep] == 0).all()
    Z.check_losses()
    assert total[0] <= 1.05 * total[1] + 1e-5 and total[2] <= 1.05 * total[3] + 1e-5, total


@pytest.mark.parametrize("t,d,v", [(1, 4096, 500), (3, 536, 821), (4, 4096, 500), (5, 4096, 500), (40, 4096, 700), (300, 2056, 700)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_loss_slopes_of_likely_targets(t, d, v, dtype):
    """A target of probability 0.999 has a slope of 0.001: what its logit and lse are off counts a thousandfold.

    The bound on a slope: up to four tokens float sums in lanes, 2^-22 of the logit for it, lse and their rounding
    each; beyond, lse comes from parts of up to 512 products, 34 steps of at most 2^-23.  Besides, the rounding of
    the slopes and of the result, each as large as e, that of the exact gradients.
    """
    gen = seeded(t, d, v)
    w = rows_of(gen, v, d, dtype, 0.05)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    high = math.log(v) + 6.9
    h = (0.2 * torch.randn(t, d, generator=gen, device="cuda") + high * w[y].float() / w[y].float().square().sum(1, keepdim=True)).to(dtype)
    g = torch.ones(t, device="cuda")
    z, lse64, _, counts, at = loss64(h, w, y)
    q = torch.exp(z - lse64[:, None])
    rows = torch.arange(t, device="cuda")
    q[rows, y] = torch.expm1(z[rows, y] - lse64)
    off = (3 * 2.0 ** -22 if t <= 4 else 34 * 2.0 ** -23) * high
    gh, gw = Z.linear_loss_backward(h, w, y, Z.linear_loss(h, w, y)[1], g)
    Z.check_losses()
    for got, ref in ((gh, q @ w.double()), (gw, q.t() @ h.double())):
        e = ((ref.to(dtype).double() - ref).norm() / ref.norm()).item()
        room = 2.1 * e + off * t ** 0.5 / q[rows, y].norm().item()
        err = ((got.double() - ref).norm() / ref.norm()).item()
        assert err <= room, (err, room)


def test_loss_more_than_one_piece():
    """So many tokens that the slopes take the vocabulary in pieces."""
    t, d, v = 3100, 64, 50257
    need = Z.zero_loss_workspace(t, v, d)[1]
    assert need < t * v * 2
    check_loss(*case(t, d, v, BF, 0.1))


def test_loss_peaked_logits():
    """Targets whose probability is near 1, and logits far apart."""
    t, d, v = 200, 768, 3001
    h, w, y, g = case(t, d, v, BF)
    h = (h.float() + 40.0 * torch.rand(t, 1, device="cuda") * w[y].float() / (0.05 ** 2 * d)).to(BF)
    check_loss(h, w, y, g)
    check_loss((h * 8).to(FP), w.to(FP), y, g)


@pytest.mark.parametrize("t", [3, 40])
def test_loss_masked_places_hold_anything(t):
    """An ignored token's hidden state may hold NaN and infinities: no gradient knows of it."""
    h, w, y, g = case(t, 264, 999, FP)
    bad = torch.arange(t, device="cuda") % 3 == 1
    y = torch.where(bad, -100, y)
    clean = torch.where(bad[:, None], 0.0, h.float()).to(FP)
    loss, lse, gh, gw = check_loss(clean, w, y, g)
    h[bad] = float("nan")
    h[bad, 0] = float("inf")
    g[bad] = float("nan")
    loss2, lse2 = Z.linear_loss(h, w, y)
    assert torch.equal(loss, loss2) and torch.equal(lse[~bad], lse2[~bad])
    gh2, gw2 = Z.linear_loss_backward(h, w, y, lse2, g)
    assert torch.equal(gh, gh2) and torch.equal(gw, gw2)
    Z.check_losses()


@pytest.mark.parametrize("t", [2, 300])
def test_loss_rows_do_not_touch_each_other(t):
    h, w, y, g = case(t, 136, 600, BF)
    loss, lse = Z.linear_loss(h, w, y)
    gh, _ = Z.linear_loss_backward(h, w, y, lse, g)
    h[1, 5] = float("nan")
    loss2, lse2 = Z.linear_loss(h, w, y)
    gh2, gw2 = Z.linear_loss_backward(h, w, y, lse2, g)
    rest = torch.arange(t, device="cuda") != 1
    assert torch.equal(loss[rest], loss2[rest]) and loss2[1].isnan() and lse2[1].isnan()
    assert torch.equal(gh[rest], gh2[rest]) and gh2[1].isnan().all() and gw2.isnan().any()


def test_loss_infinite_logits():
    """Hidden states that make logits of -inf leave the finite ones' loss; a row of only -inf has lse -inf."""
    w = torch.zeros(300, 64, dtype=BF, device="cuda")
    w[:200, 0] = -1.0
    w[200:, 1] = 1.0
    h = torch.zeros(6, 64, dtype=BF, device="cuda")
    h[:, 0] = 3e38
    w[:200, 0] = -3e38                                   # the first 200 logits are -inf
    y = torch.tensor([250, 250, 299, 200, 250, 10], device="cuda")
    loss, lse = Z.linear_loss(h, w, y)
    assert torch.allclose(lse, torch.full_like(lse, math.log(100)), atol=1e-5)
    assert torch.allclose(loss[:5], torch.full_like(loss[:5], math.log(100)), atol=1e-5) and loss[5] == float("inf")
    few, _ = Z.linear_loss(h[:2].contiguous(), w, y[:2])
    assert torch.allclose(few, loss[:2], atol=1e-5)
    gh, gw = Z.linear_loss_backward(h[:5].contiguous(), w, y[:5], lse[:5], torch.ones(5, device="cuda"))
    # the -inf logits have probability 0; every slope is finite
    ref = torch.full((5, 300), 0.0, device="cuda", dtype=torch.float64)
    ref[:, 200:] = 0.01
    ref[torch.arange(5), y[:5]] -= 1.0
    assert torch.allclose(gh[:, 1].double(), (ref @ w.double())[:, 1], atol=1e-2)
    all_low, low_lse = Z.linear_loss(h[:5].contiguous(), w[:200].contiguous(), y[:5] % 200)
    assert (low_lse == float("-inf")).all() and all_low.isnan().all()


def test_loss_targets_outside_the_vocabulary():
    h, w, y, g = case(300, 64, 100, BF)
    Z.check_losses()
    y[7], y[200] = 100, -5
    loss, lse = Z.linear_loss(h, w, y)
    assert loss[7].isnan() and loss[200].isnan() and loss.isnan().sum() == 2
    with pytest.raises(Z.ZeroError) as e:
        Z.check_losses()
    assert e.value.code == Z.ZERO_EINVAL
    Z.check_losses()                                     # reported once
    gh, gw = Z.linear_loss_backward(h, w, y, lse, g)
    assert (gh[7] == 0).all() and (gh[200] == 0).all() and gw.isfinite().all()
    with pytest.raises(Z.ZeroError):
        Z.check_losses()
    y3 = y.clone()
    y3[7] = y3[200] = -100
    gh3, gw3 = Z.linear_loss_backward(h, w, y3, lse, g)
    assert torch.equal(gh, gh3) and torch.equal(gw, gw3)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_loss_upstream_gradients(dtype):
    """Zero, of very different sizes, larger than fp16 holds, and not finite."""
    h, w, y, g = case(300, 136, 700, dtype)
    gh, gw = Z.linear_loss_backward(h, w, y, Z.linear_loss(h, w, y)[1], torch.zeros_like(g))
    assert (gh == 0).all() and (gw == 0).all()
    check_loss(h, w, y, g * 1e-30 if dtype == BF else g * 1e-3)
    g2 = g.clone()
    g2[::2] *= 1e-4
    check_loss(h, w, y, g2)
    if dtype == BF:
        check_loss(h, w, y, g * 1e8)
    lse = Z.linear_loss(h, w, y)[1]
    ref, _ = Z.linear_loss_backward(h, w, y, lse, g)
    g[3] = float("inf")
    gh, gw = Z.linear_loss_backward(h, w, y, lse, g)
    rest = torch.arange(300, device="cuda") != 3
    assert gh[rest].isfinite().all() and not gh[3].isfinite().all() and not gw.isfinite().all()
    assert torch.allclose(gh[rest].float(), ref[rest].float(), rtol=2 ** -7 if dtype == BF else 2 ** -9, atol=1e-5)


def test_loss_no_tokens():
    h, w, y, g = case(0, 64, 300, BF)
    loss, lse = Z.linear_loss(h, w, y)
    assert loss.shape == (0,) and lse.shape == (0,)
    gw = torch.full((300, 72), 3.0, dtype=BF, device="cuda")
    gh, out = Z.linear_loss_backward(h, w, y, lse, g, grad_weight=gw[:, :64])
    assert gh.shape == (0, 64) and (gw[:, :64] == 0).all() and (gw[:, 64:] == 3).all()


@pytest.mark.parametrize("t", [4, 301])
def test_loss_outputs_stay_in_their_rows(t):
    """Gradients written into parts of wider buffers leave the rest alone."""
    h, w, y, g = case(t, 200, 333, FP, 0.2, 24)
    loss, lse = Z.linear_loss(h, w, y)
    ref = Z.linear_loss_backward(h, w, y, lse, g)
    wide_h = torch.full((t + 2, 216), 5.0, dtype=FP, device="cuda")
    wide_w = torch.full((335, 208), 5.0, dtype=FP, device="cuda")
    got = Z.linear_loss_backward(h, w, y, lse, g, grad_hidden=wide_h[1:-1, 8:208], grad_weight=wide_w[1:-1, :200])
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert (wide_h[0] == 5).all() and (wide_h[-1] == 5).all() and (wide_h[:, :8] == 5).all() and (wide_h[:, 208:] == 5).all()
    assert (wide_w[0] == 5).all() and (wide_w[-1] == 5).all() and (wide_w[:, 200:] == 5).all()


def test_loss_streams_graphs_and_repeats():
    h, w, y, g = case(700, 264, 5000, BF, 0.1)
    loss, lse = Z.linear_loss(h, w, y)
    gh, gw = Z.linear_loss_backward(h, w, y, lse, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (None, side, int(side.cuda_stream)):
        l2, e2 = Z.linear_loss(h, w, y, stream=s)
        a, b = Z.linear_loss_backward(h, w, y, e2, g, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(l2, loss) and torch.equal(a, gh) and torch.equal(b, gw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l3, e3 = Z.linear_loss(h, w, y)
        a3, b3 = Z.linear_loss_backward(h, w, y, e3, g)
    for _ in range(2):
        l3.zero_()
        a3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(l3, loss) and torch.equal(a3, gh) and torch.equal(b3, gw)
    h2 = rows_of(seeded(5), 700, 264, BF)
    h.copy_(h2)
    graph.replay()
    torch.cuda.synchronize()
    l4, e4 = Z.linear_loss(h2, w, y)
    assert torch.equal(l3, l4)


def test_loss_against_differences():
    """The gradients against central differences of the 64-bit loss."""
    h, w, y, g = case(9, 40, 50, FP, 0.2)
    loss, lse = Z.linear_loss(h, w, y)
    gh, gw = Z.linear_loss_backward(h, w, y, lse, g)

    def value(H, W):
        z = H @ W.t()
        at = torch.where(y >= 0, y, 0)
        each = torch.logsumexp(z, 1) - z.gather(1, at[:, None])[:, 0]
        return (torch.where(y >= 0, each, 0.0) * g.double()).sum().item()

    H, W, step = h.double(), w.double(), 1e-5
    u, least = half_ulp(FP)
    for k in range(30):
        d = torch.zeros_like(H)
        i, j = k % 9, (k * 7) % 40
        d[i, j] = step
        slope = (value(H + d, W) - value(H - d, W)) / (2 * step)
        # the result's rounding, and that of the slopes: u of each term
        terms = 2 * g[i].abs().item() * W[:, j].abs().max().item()
        assert abs(gh[i, j].item() - slope) <= u * (abs(slope) + terms) * 1.01 + least + 1e-6
        e = torch.zeros_like(W)
        v = (k * 11) % 50
        e[v, j] = step
        slope = (value(H, W + e) - value(H, W - e)) / (2 * step)
        q = torch.softmax(H @ W.t(), 1)[:, v] - (y == v).double()
        terms = (q * g.double() * H[:, j]).abs().sum().item()
        assert abs(gw[v, j].item() - slope) <= u * (abs(slope) + terms) * 1.01 + least + 1e-6


def test_loss_wait_that_runs_out():
    """A wait that gives up at once ends the kernels, sets the status, and is reported once."""
    h, w, y, g = case(300, 768, 2000, BF)
    loss, lse = Z.linear_loss(h, w, y)
    gh, gw = Z.linear_loss_backward(h, w, y, lse, g)
    Z.check_losses()
    Z.zero_loss_set_wait_limit(0)
    try:
        Z.linear_loss(h, w, y)
        with pytest.raises(Z.ZeroError) as e:
            Z.check_losses()
        assert e.value.code == Z.ZERO_ETIMEOUT
        Z.linear_loss_backward(h, w, y, lse, g)
        with pytest.raises(Z.ZeroError) as e:
            Z.check_losses()
        assert e.value.code == Z.ZERO_ETIMEOUT
    finally:
        Z.zero_loss_set_wait_limit(4_000_000_000)
    l2, e2 = Z.linear_loss(h, w, y)
    a, b = Z.linear_loss_backward(h, w, y, lse, g)
    Z.check_losses()
    assert torch.equal(l2, loss) and torch.equal(a, gh) and torch.equal(b, gw)


@pytest.mark.parametrize("t", [2, 5])
def test_loss_offsets_beyond_32_bits(t):
    """A matrix of more than 2^31 elements: only its last rows are not zero."""
    v, d = 140000, 16384
    w = torch.zeros(v, d, dtype=BF, device="cuda")
    gen = seeded(98)
    w[-3:] = rows_of(gen, 3, d, BF, 0.02)
    h = rows_of(gen, t, d, BF)
    y = torch.full((t,), v - 2, device="cuda")
    loss, lse = Z.linear_loss(h, w, y)
    z = h.double() @ w[-3:].double().t()
    ref = torch.log(z.exp().sum(1) + (v - 3))
    ez = logit_error(h, w[-3:])
    assert ((lse.double() - ref).abs() <= ez + 4e-6 + ref * 2.0 ** -23).all()
    assert ((loss.double() - (ref - z[:, 1])).abs() <= 2 * ez + 8e-6 + ref * 2.0 ** -23).all()
    g = torch.ones(t, device="cuda")
    gh, gw = Z.linear_loss_backward(h, w, y, lse, g)
    q = torch.exp(z - ref[:, None])
    q[:, 1] -= 1
    u, _ = half_ulp(BF)
    err = q.abs() * (u * 1.01 + 1e-4)
    close(gw[-3:], q.t() @ h.double(), BF, err.t() @ h.double().abs())
    close(gh, q @ w[-3:].double(), BF, (q.abs() * (u * 1.01 + 1e-4)) @ w[-3:].double().abs())
    flat = torch.exp(-ref)
    q0 = flat[None, :].expand(2, t)
    close(gw[:2], q0 @ h.double(), BF, (q0 * (u * 1.01 + 1e-4)) @ h.double().abs())
    Z.check_losses()


# ---- global norm, clipping, packing -----------------------------------------------------

def clip64(grads, max_norm, scale):
    total = math.fsum(g.double().square().sum().item() for g in grads)
    norm = math.sqrt(total) / scale
    return norm, min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0


def check_clip(grads, flat, offsets, got, max_norm, scale):
    norm, coef = clip64(grads, max_norm, scale)
    n, c, bad = got
    # chunks in float (at most 64 squares a sum, 2^-24 each), doubles above, rounded once
    assert abs(n.item() - norm) <= norm * 20 * 2.0 ** -24 + 2.0 ** -149
    assert abs(c.item() - coef) <= coef * 24 * 2.0 ** -24
    assert bad.item() == 0
    for g, o in zip(grads, offsets):
        out = flat[o:o + g.numel()]
        ref = g.double() * c.double()
        if g.dtype == torch.float32:
            assert ((out.double() - ref).abs() <= ref.abs() * 2.0 ** -24 + 2.0 ** -150).all()
        else:
            close(out, ref, g.dtype, ref.abs() * 2.0 ** -23)


def tensors(gen, lens, dtype, std, shift):
    """Gradients that start `shift` elements into their storage."""
    return [(torch.randn(n + shift, generator=gen, device="cuda") * std).to(dtype)[shift:] for n in lens]


@pytest.mark.parametrize("dtype", [BF, FP, torch.float32])
@pytest.mark.parametrize("lens", [[1], [7], [8], [9, 1, 0, 15], [0, 0, 3], [16384], [16385, 16383, 5], [100000, 33, 1 << 20],
                                  [3] * 700, [257, 4099] * 40])
def test_clip_packs(lens, dtype):
    gen = seeded(len(lens), sum(lens))
    for shift, lead, max_norm, scale in ((0, 0, 1.0, 1.0), (1, 3, 0.01, 1024.0), (5, 8, 0.0, 1.0), (2, 1, 1e9, 2.0)):
        std = 0.02 * (scale if dtype != FP else min(scale, 64.0))
        grads = tensors(gen, lens, dtype, std, shift)
        before = [g.clone() for g in grads]
        flat = torch.full((lead + sum(lens) + 9,), 7.0, dtype=dtype, device="cuda")
        offsets = list(np.cumsum([lead] + lens[:-1]))
        got = Z.clip_gradients(grads, flat, offsets, max_norm=max_norm, loss_scale=scale)
        check_clip(grads, flat, offsets, got, max_norm, scale)
        assert (flat[:lead] == 7).all() and (flat[lead + sum(lens):] == 7).all()
        assert all(torch.equal(a, b) for a, b in zip(before, grads))
        again = Z.clip_gradients(grads, flat, offsets, max_norm=max_norm, loss_scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        # a list of outputs, and in place: the same bits
        outs = [torch.empty_like(g) for g in grads]
        third = Z.clip_gradients(grads, outs, max_norm=max_norm, loss_scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(got, third))
        fourth = Z.clip_gradients(grads, max_norm=max_norm, loss_scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(got, fourth))
        for g, o, at, n in zip(grads, outs, offsets, lens):
            assert torch.equal(g, o) and torch.equal(g, flat[at:at + n])


def test_clip_into_a_plans_layout():
    """The flat buffer of a plan whose tensors have odd lengths, ready for its reduce."""
    lens = [1001, 17, 30001, 3]
    plan = Z.ZeroPlan(-1, 2, lens, 128, 1, None, Z.ZERO_BF16)
    gen = seeded(3)
    grads = tensors(gen, lens, BF, 0.1, 0)
    flat = torch.zeros(plan.psi_padded, dtype=BF, device="cuda")
    got = Z.clip_gradients(grads, flat, plan.tensor_offsets, max_norm=1.0)
    check_clip(grads, flat, plan.tensor_offsets, got, 1.0, 1.0)
    assert (flat[sum(lens):] == 0).all()
    P = plan.part_len
    for r in range(2):
        out = torch.empty(P, device="cuda")
        plan.reduce(r, [flat[r * P:(r + 1) * P]] * 2, out, 1.0)
        assert torch.equal(out, flat[r * P:(r + 1) * P].float())
    plan.close()


@pytest.mark.parametrize("dtype,values", [
    (torch.float32, [1e30, 1e-30, 3e38]), (BF, [1e30, 1e-30, 3e38]), (FP, [65504.0, 6e-8, 6e-8]),
    (torch.float32, [1e-42, 1e-44, 0.0]), (torch.float32, [1e-25, 1e-25, 1e-25])])
def test_clip_extremes(dtype, values):
    """Squares that leave float's range in either direction."""
    grads = [torch.full((n,), v, dtype=dtype, device="cuda") for n, v in zip((5, 40001, 3), values)]
    norm, coef, bad = Z.clip_gradients(grads, torch.empty(40009, dtype=dtype, device="cuda"), max_norm=1.0)
    ref, c = clip64(grads, 1.0, 1.0)
    # a norm beyond float is reported as infinity; the coefficient is decided in double
    assert norm.item() == float("inf") if ref > 3.4028235e38 else abs(norm.item() - ref) <= ref * 20 * 2.0 ** -24 + 2.0 ** -150
    assert abs(coef.item() - c) <= c * 24 * 2.0 ** -24 + 2.0 ** -150 and bad.item() == 0


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF, FP, torch.float32])
def test_clip_not_finite(dtype, value):
    """One element that is not finite: the flag, and gradients as they were."""
    for n, at in ((3, 2), (100001, 0), (100001, 100000), (100001, 50000)):
        grads = tensors(seeded(n), [n, 40], dtype, 1.0, 1)
        grads[0][at] = value
        flat = torch.zeros(n + 40, dtype=dtype, device="cuda")
        norm, coef, bad = Z.clip_gradients(grads, flat, max_norm=0.5)
        assert bad.item() == 1 and coef.item() == 1.0 and not math.isfinite(norm.item())
        whole = torch.cat(grads)
        assert torch.equal(flat.isnan(), whole.isnan()) and torch.equal(flat[~whole.isnan()], whole[~whole.isnan()])


def test_clip_zeros_and_nothing():
    zero = [torch.zeros(70000, dtype=BF, device="cuda"), torch.zeros(0, dtype=BF, device="cuda")]
    norm, coef, bad = Z.clip_gradients(zero, torch.empty(70000, dtype=BF, device="cuda"), max_norm=1.0)
    assert norm.item() == 0 and coef.item() == 1 and bad.item() == 0
    norm, coef, bad = Z.clip_gradients([zero[1]], torch.empty(0, dtype=BF, device="cuda"), max_norm=1.0)
    assert norm.item() == 0 and coef.item() == 1 and bad.item() == 0
    # norm only, by the C call
    g = torch.full((9,), 2.0, device="cuda")
    found = torch.zeros(3, device="cuda")
    space = torch.empty(4096, dtype=torch.uint8, device="cuda")
    Z.zero_clip_gradients([g], [9], Z.ZERO_FP32, None, 1.0, 3.0, found, None, None, space, 4096)
    assert found.tolist() == [6.0, 0.0, 0.0]


def test_clip_streams_and_graphs():
    lens = [40001, 3, 70000] * 10
    grads = tensors(seeded(8), lens, FP, 1.0, 0)
    flat = torch.zeros(sum(lens), dtype=FP, device="cuda")
    got = [x.clone() for x in Z.clip_gradients(grads, flat, max_norm=1.0)]
    ref = flat.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    flat.zero_()
    torch.cuda.synchronize()
    two = Z.clip_gradients(grads, flat, max_norm=1.0, stream=side)
    side.synchronize()
    assert torch.equal(flat, ref) and all(torch.equal(a, b) for a, b in zip(got, two))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        three = Z.clip_gradients(grads, flat, max_norm=1.0)
    flat.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(flat, ref) and all(torch.equal(a, b) for a, b in zip(got, three))


def test_clip_offsets_beyond_32_bits():
    n = (1 << 31) + 12345
    g = torch.full((n,), 2.0, dtype=BF, device="cuda")
    g[-1] = 3.0
    flat = torch.empty(n + 1, dtype=BF, device="cuda")
    norm, coef, bad = Z.clip_gradients([g], flat, [1], max_norm=1.0)
    ref = math.sqrt(4.0 * (n - 1) + 9.0)
    assert abs(norm.item() - ref) <= ref * 20 * 2.0 ** -24 and bad.item() == 0
    two, three = (torch.tensor([2.0, 3.0], device="cuda") * coef).to(BF)
    assert flat[-1] == three and (flat[1:-1] == two).all()


# ---- refusals of the tensor functions ------------------------------------------------------

def test_head_refuses():
    gen = seeded(1)
    x, w = rows_of(gen, 4, 64, BF), rows_of(gen, 1, 64, BF)[0].contiguous()
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    lse = f
    vocab = rows_of(gen, 10, 64, BF)
    for call in (
        lambda: Z.residual_norm(x.float(), None, w, EPS), lambda: Z.residual_norm(x.cpu(), None, w, EPS),
        lambda: Z.residual_norm(x, x[:2], w, EPS), lambda: Z.residual_norm(x, x.half(), w, EPS),
        lambda: Z.residual_norm(x, None, w.half(), EPS), lambda: Z.residual_norm(x, None, w[:8], EPS),
        lambda: Z.residual_norm(x.t(), None, w, EPS), lambda: Z.residual_norm(x[0], None, w, EPS),
        lambda: Z.residual_norm(x, None, w, -1.0), lambda: Z.residual_norm_quantized(x, None, w, EPS, 5),
        lambda: Z.residual_norm(x[:, :60], None, w[:60], EPS), lambda: Z.residual_norm(x[:, 4:60], None, w[:56], EPS),
        lambda: Z.dequantize_rows(x, f, 0, BF), lambda: Z.dequantize_rows(torch.zeros(4, 64, dtype=torch.int8, device="cuda"), f, 0, BF),
        lambda: Z.residual_norm_backward(x, w, x[:, :8], None, EPS), lambda: Z.residual_norm_backward(x, w, x, x.half(), EPS),
        lambda: Z.linear_loss(x, vocab.half(), y), lambda: Z.linear_loss(x, vocab[:, :8], y), lambda: Z.linear_loss(x, vocab, y[:3]),
        lambda: Z.linear_loss(x, vocab, y.int()), lambda: Z.linear_loss(x, vocab, y.cpu()), lambda: Z.linear_loss(x, vocab[:0], y),
        lambda: Z.linear_loss_backward(x, vocab, y, lse[:2], f), lambda: Z.linear_loss_backward(x, vocab, y, lse, f.double()),
        lambda: Z.linear_loss_backward(x, vocab, y, lse, f, grad_hidden=x[:2]),
        lambda: Z.linear_loss_backward(x, vocab, y, lse, f, grad_weight=vocab.half()),
        lambda: Z.clip_gradients([]), lambda: Z.clip_gradients([x, x.half()]), lambda: Z.clip_gradients([x.cpu()]),
        lambda: Z.clip_gradients([x.t()]), lambda: Z.clip_gradients([y]), lambda: Z.clip_gradients([x], x),
        lambda: Z.clip_gradients([x], torch.zeros(255, dtype=BF, device="cuda")),
        lambda: Z.clip_gradients([x], torch.zeros(300, dtype=BF, device="cuda"), [45]),
        lambda: Z.clip_gradients([x], torch.zeros(300, dtype=BF, device="cuda"), [-1]),
        lambda: Z.clip_gradients([x], torch.zeros(300, dtype=BF, device="cuda"), [0, 1]),
        lambda: Z.clip_gradients([x], [x, x]), lambda: Z.clip_gradients([x], [x[:2]]), lambda: Z.clip_gradients([x], max_norm=float("nan")),
        lambda: Z.clip_gradients([x], loss_scale=0.0),
    ):
        with pytest.raises(Z.ZeroError) as e:
            call()
        assert e.value.code in (Z.ZERO_EINVAL, Z.ZERO_EALIGN)
