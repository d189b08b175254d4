"""The gated projections and their gradients on the GPU, against 64-bit torch.

Tolerances, element by element, from what is rounded (half(t) is half a step of type t, relative):
  g, u      float sums of D products in the tensor core: each 16 products drop up to 2^-22 of the largest partial sum
            (2^-23 in bf16), which the sum of magnitudes S bounds: (D / 16 + 4) 2^-22 S
  act       P by an exponential whose argument y is off by 2^-23 |y|, one approximate reciprocal and three
            products: (|y| + 16) 2^-22 relative, where y = g, 2y of the tanh, or g^2 / 2
  out       rounded once: half(t) of itself, half of t's smallest step below that
  dg, du    rounded to t for the products: half(t) each (fp16 scaled: an absolute 2^-23 of the largest |grad_out| besides),
            carried to the gradients by the products' magnitudes; the sums of the products as for g; the result's rounding
"""
import math

import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
ACTS = ["silu", "gelu", "gelu_tanh"]
UNIT = 2.0 ** -22


def half(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Half of the type's smallest step."""
    return 2.0 ** -25 if dtype == FP else 2.0 ** -134


def rows_of(gen, rows, cols, dtype, std=1.0, pad=0):
    return (torch.randn(rows, cols + pad, generator=gen, device="cuda") * std).to(dtype)[:, :cols]


def case(t, d, f, dtype, pad=0, key=0, std=0.1):
    gen = torch.Generator(device="cuda").manual_seed(hash((t, d, f, key)) % (1 << 31))
    return (rows_of(gen, t, d, dtype, 1.0, pad), rows_of(gen, f, d, dtype, std, pad), rows_of(gen, f, d, dtype, std, pad),
            rows_of(gen, t, f, dtype, 1e-2, pad))


def share(act, g):
    """(P, P', the argument's size): the activation is g P."""
    if act == "silu":
        p = torch.sigmoid(g)
        return p, p * torch.sigmoid(-g), g.abs()
    if act == "gelu":
        return 0.5 * torch.erfc(-g / math.sqrt(2)), torch.exp(-g * g / 2) / math.sqrt(2 * math.pi), g * g / 2
    c = math.sqrt(2 / math.pi)
    y = 2 * c * (g + 0.044715 * g ** 3)
    p = torch.sigmoid(y)
    return p, p * torch.sigmoid(-y) * 2 * c * (1 + 3 * 0.044715 * g * g), y.abs()


class Exact:
    """Everything in 64 bits, with the errors that are allowed."""

    def __init__(self, x, gate, up, act, grad=None):
        dtype = x.dtype
        t, d = x.shape
        x, gate, up = x.double(), gate.double(), up.double()
        steps = (d / 16 + 4) * UNIT
        g, u = x @ gate.T, x @ up.T
        eg, eu = steps * (x.abs() @ gate.abs().T), steps * (x.abs() @ up.abs().T)
        p, dp, y = share(act, g)
        ep = (y + 16) * UNIT * p
        a, slope = g * p, p + g * dp
        # act' and its derivative are below 1.2 in all three
        ea = 1.2 * eg + g.abs() * ep
        eslope = 1.2 * eg + ep + g.abs() * dp.abs() * (y + 16) * 2 * UNIT + 4 * UNIT * p
        self.out = a * u
        self.out_off = half(dtype) * self.out.abs() + floor_of(dtype) + 1.01 * (ea * u.abs() + a.abs() * eu + 4 * UNIT * self.out.abs())
        if grad is None:
            return
        go = grad.double()
        finite = go.abs()[torch.isfinite(go)]
        top = float(finite.max()) if finite.numel() else 0.0
        tiny = 2.0 ** -23 * top if dtype == FP else 2.0 ** -134
        dg, du = go * u * slope, go * a
        edg = half(dtype) * dg.abs() + tiny + 1.01 * go.abs() * (eu * slope.abs() + u.abs() * eslope + 4 * UNIT * (u * slope).abs())
        edu = half(dtype) * du.abs() + tiny + 1.01 * go.abs() * (ea + 4 * UNIT * a.abs())
        f = gate.shape[0]
        sums = lambda n: (n / 16 + 20) * UNIT  # noqa: E731
        self.gx = dg @ gate + du @ up
        size = dg.abs() @ gate.abs() + du.abs() @ up.abs()
        self.gx_off = half(dtype) * self.gx.abs() + floor_of(dtype) + 1.01 * (edg @ gate.abs() + edu @ up.abs() + sums(2 * f) * size)
        self.gg, self.gu = dg.T @ x, du.T @ x
        self.gg_off, self.gu_off = (
            half(dtype) * ref.abs() + floor_of(dtype) + 1.01 * (e.T @ x.abs() + sums(t) * (s.abs().T @ x.abs()))
            for ref, e, s in ((self.gg, edg, dg), (self.gu, edu, du)))


def near(got, ref, off):
    far = (got.double() - ref).abs() > off
    assert not far.any(), (int(far.sum()), got[far][:4], ref[far][:4], off[far][:4])


def check(x, gate, up, grad, act, seen=None):
    e = Exact(x, gate, up, act, grad)
    out = Z.gated_linear(x, gate, up, act)
    near(out, e.out, e.out_off)
    gx, gg, gu = Z.gated_linear_backward(x, gate, up, grad, act)
    near(gx, e.gx, e.gx_off)
    near(gg, e.gg, e.gg_off)
    near(gu, e.gu, e.gu_off)
    Z.check_losses()
    return out, gx, gg, gu


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("t,d,f", [(1, 8, 8), (2, 72, 136), (3, 64, 24), (5, 264, 40), (33, 136, 264), (129, 520, 128),
                                   (257, 72, 520)])
def test_small(t, d, f, dtype, act):
    check(*case(t, d, f, dtype, pad=8 if t % 2 else 0), act)


@pytest.mark.parametrize("t,d,f,dtype,act", [
    (1, 4096, 1000, BF, "silu"), (4, 1600, 4264, FP, "gelu"), (7, 1600, 264, BF, "gelu_tanh"), (48, 1600, 4264, BF, "silu"),
    (300, 4088, 72, FP, "silu"), (64, 4096, 4264, BF, "gelu"), (65, 1600, 136, FP, "silu"), (16, 768, 11000, FP, "gelu_tanh"),
    (31, 16384, 136, BF, "silu"), (100, 4088, 400, BF, "gelu"), (128, 4096, 1000, FP, "silu"), (70, 2000, 136, FP, "gelu_tanh"), (1, 200, 40000, BF, "silu"), (1023, 768, 2048, BF, "gelu"), (2100, 72, 1352, FP, "gelu_tanh"), (513, 264, 5000, BF, "silu"),
])
def test_larger(t, d, f, dtype, act):
    check(*case(t, d, f, dtype, std=0.03), act)


@pytest.mark.parametrize("t", [1, 3, 40, 300])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_halves_of_one_matrix_and_interleaved_rows(t, dtype):
    x, _, _, grad = case(t, 72, 136, dtype)
    gen = torch.Generator(device="cuda").manual_seed(5)
    both = rows_of(gen, 272, 72, dtype, 0.1)
    check(x, both[:136], both[136:], grad, "silu")
    check(x, both[0::2], both[1::2], grad, "silu")


@pytest.mark.parametrize("t", [2, 70])
@pytest.mark.parametrize("dtype,size", [(FP, 2.0 ** -20), (FP, 3e4), (BF, 1e-30), (BF, 1e30)])
def test_gradients_of_any_size(t, dtype, size):
    """fp16 slopes would leave its range unscaled; the results themselves fit."""
    x, gate, up, _ = case(t, 136, 72, dtype)
    gen = torch.Generator(device="cuda").manual_seed(6)
    grad = (torch.rand(t, 72, generator=gen, device="cuda") * 2 - 1).mul_(size).to(dtype)
    if dtype == FP and size > 1:
        x, gate, up = x * 0.01, gate * 0.01, up * 0.01
    check(x, gate, up, grad, "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t", [1, 4, 130])
def test_far_arguments(t, act):
    """Activations far out on both sides: no overflow on the way, and the right zeros."""
    gate = torch.zeros(72, 8, device="cuda", dtype=BF)
    gate[:, 0] = torch.linspace(-1, 1, 72, device="cuda").mul(120).to(BF)
    up = torch.full((72, 8), 0.5, device="cuda", dtype=BF)
    x = torch.zeros(t, 8, device="cuda", dtype=BF)
    x[:, 0] = torch.tensor([1.0, 8.0, 0.1, 1000.0], device="cuda").to(BF).repeat(t)[:t]
    grad = torch.ones(t, 72, device="cuda", dtype=BF)
    out, gx, gg, gu = check(x, gate, up, grad, act)
    for r in (out, gx, gg, gu):
        assert torch.isfinite(r).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("t", [3, 60])
def test_rows_without_gradient_and_zero_rows(t, dtype):
    x, gate, up, grad = case(t, 72, 136, dtype)
    x, grad = x.clone(), grad.clone()
    grad[1::2] = 0
    x[0] = 0
    _, gx, _, _ = check(x, gate, up, grad, "silu")
    assert (gx[1::2] == 0).all()
    grad.zero_()
    _, gx, gg, gu = check(x, gate, up, grad, "silu")
    for r in (gx, gg, gu):
        assert (r == 0).all()


@pytest.mark.parametrize("t", [3, 4, 60])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_do_not_touch_each_other(t, bad):
    x, gate, up, grad = case(t, 72, 136, FP)
    out = Z.gated_linear(x, gate, up)
    gx, _, _ = Z.gated_linear_backward(x, gate, up, grad)
    x2, grad2 = x.clone(), grad.clone()
    x2[1, 5] = bad
    grad2[2, 7] = bad
    out2 = Z.gated_linear(x2, gate, up)
    gx2, gg2, gu2 = Z.gated_linear_backward(x2, gate, up, grad2)
    keep = [i for i in range(t) if i != 1]
    assert torch.equal(out2[keep], out[keep]) and not torch.isfinite(out2[1]).any()
    keep = [i for i in range(t) if i not in (1, 2)]
    assert torch.equal(gx2[keep], gx[keep])
    assert not torch.isfinite(gx2[2]).any()
    assert not torch.isfinite(gg2[7]).any() and not torch.isfinite(gu2[7]).any()


@pytest.mark.parametrize("left", [0, 8, 16])
@pytest.mark.parametrize("t,d,f", [(1, 72, 136), (3, 264, 72), (40, 72, 136), (300, 520, 264), (300, 8, 8)])
def test_outputs_stay_in_their_rows(t, d, f, left):
    """Output rows that are parts of wider ones, some of them off the sectors of 32 bytes, and what stands around them."""
    x, gate, up, grad = case(t, d, f, BF)
    want = Z.gated_linear_backward(x, gate, up, grad)
    wide = [torch.full((n + 5, d + 24), 7.0, device="cuda", dtype=BF) for n in (t, f, f)]
    into = [w[:n, left:left + d] for w, n in zip(wide, (t, f, f))]
    got = Z.gated_linear_backward(x, gate, up, grad, grad_x=into[0], grad_gate=into[1], grad_up=into[2])
    for g, i, w, r, n in zip(got, into, wide, want, (t, f, f)):
        assert g.data_ptr() == i.data_ptr() and torch.equal(i, r)
        assert (w[:, :left] == 7).all() and (w[:, left + d:] == 7).all() and (w[n:] == 7).all()


@pytest.mark.parametrize("left", [0, 8])
@pytest.mark.parametrize("t,d,f", [(3, 64, 136), (70, 64, 136), (300, 64, 1000)])
def test_forward_output_stays_in_its_rows(t, d, f, left):
    """The C call's output among wider rows."""
    x, gate, up, _ = case(t, d, f, BF)
    want = Z.gated_linear(x, gate, up)
    wide = torch.full((t + 5, f + 24), 7.0, device="cuda", dtype=BF)
    status = torch.zeros(1, device="cuda", dtype=torch.int32)
    into = wide[:t, left:left + f]
    Z.zero_gated_forward(x, d, gate, d, up, d, Z.ZERO_ACT_SILU, t, f, d, Z.ZERO_BF16, into, f + 24, status, None, 0)
    assert torch.equal(into, want) and int(status) == 0
    assert (wide[:, :left] == 7).all() and (wide[:, left + f:] == 7).all() and (wide[t:] == 7).all()


def test_no_tokens():
    x, gate, up, grad = case(3, 72, 136, BF)
    out = Z.gated_linear(x[:0], gate, up)
    assert out.shape == (0, 136)
    gx, gg, gu = Z.gated_linear_backward(x[:0], gate, up, grad[:0])
    assert gx.shape == (0, 72) and (gg == 0).all() and (gu == 0).all()


@pytest.mark.parametrize("t", [1, 4, 40, 300])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_repeats_streams_and_graphs(t, dtype):
    """The same bits from run to run, on another stream, and from two graphs replayed at once, each with its own scratch."""
    cases = [case(t, 264, 520, dtype, key=k) for k in (1, 2)]
    want = [(Z.gated_linear(*c[:3]), *Z.gated_linear_backward(*c)) for c in cases]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = (Z.gated_linear(*cases[0][:3], stream=side), *Z.gated_linear_backward(*cases[0], stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for c, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append((Z.gated_linear(*c[:3]), *Z.gated_linear_backward(*c)))
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    Z.check_losses()


@pytest.mark.parametrize("act", ACTS)
def test_against_differences(act):
    """Directional derivatives of sum(grad * out), by central differences of the 64-bit formula at the same inputs, where
    the library's gradients are rounded sums: each to within its own tolerance along the direction."""
    x, gate, up, grad = case(6, 24, 40, FP)
    got = Z.gated_linear_backward(x, gate, up, grad, act)
    e = Exact(x, gate, up, act, grad)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def value(*at):
        g = at[0] @ at[1].T
        return (grad.double() * (g * share(act, g)[0] * (at[0] @ at[2].T))).sum()

    at = [x.double(), gate.double(), up.double()]
    for k, off in enumerate((e.gx_off, e.gg_off, e.gu_off)):
        step = torch.randn(at[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        high, low = ([a + s * h * step if i == k else a for i, a in enumerate(at)] for s in (1, -1))
        slope = (value(*high) - value(*low)) / (2 * h)
        # central differences are off by h^2 / 6 of the third derivative along the step: far below
        assert abs(float(slope - (got[k].double() * step).sum())) <= float((off * step.abs()).sum()) + 1e-7


@pytest.mark.parametrize("t,d", [(300, 264), (40, 520), (3, 64)])
def test_a_wait_that_runs_out_is_reported(t, d):
    x, gate, up, grad = case(t, d, 520, BF)
    want = Z.gated_linear(x, gate, up)
    Z.check_losses()
    Z.zero_loss_set_wait_limit(0)
    try:
        Z.gated_linear(x, gate, up)
        Z.gated_linear_backward(x, gate, up, grad)
        with pytest.raises(Z.ZeroError) as e:
            Z.check_losses()
        assert e.value.code == Z.ZERO_ETIMEOUT
    finally:
        Z.zero_loss_set_wait_limit(4_000_000_000)
    assert torch.equal(Z.gated_linear(x, gate, up), want)
    Z.check_losses()


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """Rows whose byte offsets pass 2^32: the last tokens of a long batch in wide rows, forward and backward."""
    t, d, f, pad = 70_000, 64, 72, 33_000
    x = torch.zeros(t, d + pad, device="cuda", dtype=BF)[:, :d]
    gen = torch.Generator(device="cuda").manual_seed(1)
    x[-300:] = rows_of(gen, 300, d, BF)
    gate, up = rows_of(gen, f, d, BF, 0.1), rows_of(gen, f, d, BF, 0.1)
    grad = torch.zeros(t, f + pad, device="cuda", dtype=BF)[:, :f]
    grad[-300:] = rows_of(gen, 300, f, BF)
    e = Exact(x[-300:], gate, up, "silu", grad[-300:])
    out = Z.gated_linear(x, gate, up)
    near(out[-300:], e.out, e.out_off)
    assert (out[:-300] == 0).all()
    gx, gg, gu = Z.gated_linear_backward(x, gate, up, grad)
    near(gx[-300:], e.gx, e.gx_off)
    near(gg, e.gg, e.gg_off + (t / 16) * UNIT * e.gg.abs())
    near(gu, e.gu, e.gu_off + (t / 16) * UNIT * e.gu.abs())
    Z.check_losses()


def test_refuses():
    x, gate, up, grad = case(3, 72, 136, BF)
    for call in (lambda: Z.gated_linear(x, gate, up, "relu"), lambda: Z.gated_linear(x, gate, up[:128]),
                 lambda: Z.gated_linear(x, gate.half(), up), lambda: Z.gated_linear(x.float(), gate, up),
                 lambda: Z.gated_linear(x[:, :64], gate, up), lambda: Z.gated_linear(x.t().contiguous().t(), gate, up),
                 lambda: Z.gated_linear(x[:1].expand(3, 72), gate, up), lambda: Z.gated_linear(x[0], gate, up),
                 lambda: Z.gated_linear(x.cpu(), gate, up), lambda: Z.gated_linear(x, gate.requires_grad_(), up),
                 lambda: Z.gated_linear_backward(x, gate, up, grad[:2]), lambda: Z.gated_linear_backward(x, gate, up, grad[:, :128]),
                 lambda: Z.gated_linear_backward(x, gate, up, grad, grad_x=grad)):
        with pytest.raises(Z.ZeroError):
            call()
        gate = gate.detach()
