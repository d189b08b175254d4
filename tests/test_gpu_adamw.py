"""AdamW over a list of tensors on the GPU, its moments in 32 and in 8 bits, against torch.

32 bits: every operation rounded on its own, so torch's float operations in the same order give the same bits.
8 bits: against 64 bits from the same codes.  The step's arithmetic is float with fused operations, an approximate root
and an approximate quotient: new moments are off by at most 8 of 2^-24 of their terms' magnitudes (the products, the
sum, and the gradient's factor before), the root by half of v's relative error and 2^-22, the update by 2^-20 of itself.
A scale is the largest magnitude times a constant: 2^-23 more.  A code has to be the neighbour that the random bits choose,
unless the value is so near the border that its own error may cross it: then either.
"""
import math

import numpy as np
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
BLOCK = 128
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
U = 2.0 ** -24
M32 = 0xFFFFFFFF


def mix(x):
    for shift, factor in ((16, 0x9E3779B1), (15, 0xB504F333), (16, 1)):
        x = ((x ^ (x >> shift)) * factor) & M32
    return x


def random16(first, n, step, seed):
    at = torch.arange(first, first + n, dtype=torch.int64, device="cuda")
    key = mix(((mix(seed & M32) + step) & M32))
    high = torch.tensor([mix((key + h) & M32) for h in range((first + n >> 32) + 1)], device="cuda")
    word = mix((at & M32) ^ high[at >> 32])
    return word & 0xFFFF, word >> 16


def lists(gen, lens, dtype=F32, std=1.0, shift=0):
    """Tensors of these lengths, `shift` elements off an allocation's start."""
    out = []
    for n in lens:
        t = torch.randn(n + shift, generator=gen, device="cuda").mul_(std).to(dtype)
        out.append(t[shift:])
    return out


def flat(tensors, offsets, dtype=torch.float64):
    out = torch.zeros(offsets[-1], dtype=dtype, device="cuda")
    for t, o in zip(tensors, offsets):
        out[o:o + t.numel()] = t.flatten()
    return out


def values(state):
    """(m, root of v, code of |m|, code of the root) in 64 bits."""
    spread = lambda s: s.double().repeat_interleave(BLOCK)  # noqa: E731
    code = state.v.long()
    root = torch.where(code >= 32, (32 + code % 32) * torch.exp2((code // 32 - 20).double()), (code % 32) * 2.0 ** -19)
    m = state.m.view(torch.float8_e4m3fn).double()
    return m * spread(state.m_scales), root * spread(state.v_scales), state.m.view(torch.uint8).long() & 127, code


def check_codes(new, off, scale, codes, bits, mantissa, low, most, root):
    """Codes of new >= 0 (known to `off`) with this scale."""
    scale = scale.double().repeat_interleave(BLOCK)
    y = torch.where(scale > 0, new / scale, 0.0)
    y_off = torch.where(scale > 0, off / scale, 0.0) + 4 * U * y
    step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** low))).clamp_min(low) - mantissa)
    exponent = torch.log2(step) + mantissa - low           # 0 below and in the first binade
    place = y / step + (bits.double() + 0.5) / 65536       # in steps of its binade
    code_at = lambda p: (p.floor() + exponent * 2 ** mantissa).long().clamp(max=most)  # noqa: E731
    near = y_off / step + 2.0 ** -20
    low_code, high_code = code_at(place - near), code_at(place + near)
    if root:
        live = (new > off) & (scale > 0)
        low_code, high_code = (torch.where(live, c.clamp_min(1), c) for c in (low_code, high_code))
    wrong = (codes < low_code) | (codes > high_code)
    assert not wrong.any(), (int(wrong.sum()), codes[wrong][:5], low_code[wrong][:5], high_code[wrong][:5], y[wrong][:5])
    # the border cases are few
    if codes.numel() > 100_000:
        assert float((low_code != high_code).double().mean()) < 1e-3


class Case:
    def __init__(self, lens, bits, grad=BF, copy=None, shift=0, key=0, std=1e-2):
        gen = torch.Generator(device="cuda").manual_seed(key + 17)
        self.lens, self.bits = lens, bits
        self.params = lists(gen, lens, F32, 0.1, shift)
        self.grads = lists(gen, lens, grad, std, shift)
        self.copies = None if copy is None else lists(gen, lens, copy, 1.0, shift)
        self.state = Z.adamw_state(self.params, bits)
        self.offsets = Z.adamw_offsets(self.params)
        self.gen = gen

    def new_grads(self, std=1e-2):
        for g in self.grads:
            g.copy_(torch.randn(g.shape, generator=self.gen, device="cuda").mul_(std * math.exp(torch.rand(1).item())))

    def step(self, check=True, seed=0, **more):
        """One step, checked element by element."""
        args = {**HYPER, **more}
        before = [t.clone() for t in self.params]
        old = Z.AdamWState(*(None if t is None else t.clone() for t in self.state))
        Z.adamw_step(self.params, self.grads, self.state, copies=self.copies, seed=seed, **args)
        if check:
            (self.check32 if self.bits == 32 else self.check8)(before, old, seed, **args)
            if self.copies is not None:
                assert all(torch.equal(c, p.to(c.dtype)) for c, p in zip(self.copies, self.params))
        return self

    def check32(self, before, old, seed, lr, beta1, beta2, eps, weight_decay, coef=None, loss_scale=1.0, skip=None):
        t = int(old.record[0]) + 1
        assert int(self.state.record[0]) == t and int(self.state.record[1]) == 0
        f = lambda x: torch.tensor(x, dtype=torch.float64).float().item()  # noqa: E731
        bc1, bc2 = (torch.tensor(1 - b ** t, device="cuda").float() for b in (beta1, beta2))
        factor = torch.tensor(1.0 / loss_scale, device="cuda") * (1.0 if coef is None else coef)
        p, g = flat(before, self.offsets, F32), flat([g.float() for g in self.grads], self.offsets, F32) * factor
        m = old.m * f(beta1) + g * f(1 - beta1)
        v = old.v * f(beta2) + (g * g) * f(1 - beta2)
        want = p * f(1 - lr * weight_decay) - ((m / bc1) * f(lr)) / ((v / bc2).sqrt() + f(eps))
        assert torch.equal(self.state.m, m) and torch.equal(self.state.v, v)
        got = flat(self.params, self.offsets, F32)
        assert torch.equal(got, want)

    def check8(self, before, old, seed, lr, beta1, beta2, eps, weight_decay, coef=None, loss_scale=1.0, skip=None):
        t = int(old.record[0]) + 1
        assert int(self.state.record[0]) == t and int(self.state.record[1]) == 0
        g = flat(self.grads, self.offsets) * (1.0 if coef is None else float(coef)) / loss_scale
        p = flat(before, self.offsets)
        m0, r0, _, _ = values(old)
        m, v = beta1 * m0 + (1 - beta1) * g, beta2 * r0 ** 2 + (1 - beta2) * g ** 2
        m_off = 8 * U * (beta1 * m0.abs() + (1 - beta1) * g.abs())
        r = v.sqrt()
        r_off = 8 * U * r + 2.0 ** -62  # v below 2^-126 is no float's normal number
        c1, c2 = 1 - beta1 ** t, 1 - beta2 ** t
        denom = r / math.sqrt(c2) + eps
        update = lr * (m / c1) / denom
        want = p * (1 - lr * weight_decay) - update
        off = 4 * U * (p.abs() + want.abs()) + 2.0 ** -20 * update.abs() + lr / c1 / denom * (m_off + m.abs() * r_off / denom / math.sqrt(c2))
        got = flat(self.params, self.offsets)
        inside = flat([torch.ones(n, device="cuda") for n in self.lens], self.offsets) > 0
        assert not (((got - want).abs() > off) & inside).any()
        bits_m, bits_r = random16(0, self.offsets[-1], t, seed)
        _, _, code_m, code_r = values(self.state)
        for new, o, scale, top in ((m.abs(), m_off, self.state.m_scales, 448.0), (r, r_off, self.state.v_scales, 1.96875 / 256)):
            rows, offs = (x.view(-1, BLOCK).amax(1) for x in (new, o))
            assert ((scale.double() * top - rows).abs() <= 4 * U * rows + offs + 2.0 ** -126).all()
        check_codes(m.abs(), m_off, self.state.m_scales, code_m, bits_m, 3, -6, 126, False)
        check_codes(r, r_off, self.state.v_scales, code_r, bits_r, 5, -14, 255, True)
        sign = self.state.m.view(torch.uint8) > 127
        assert torch.equal(sign[code_m > 0], (m < 0)[code_m > 0])
        assert (self.state.m[~inside] == 0).all() and (self.state.v[~inside] == 0).all()


LISTS = [[1], [4], [127], [128], [129, 5], [1000, 1, 3, 4096, 130], [2 ** 15 + 3], [512] * 9]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lens", LISTS, ids=lambda x: "-".join(map(str, x[:4])))
@pytest.mark.parametrize("grad,copy", [(BF, BF), (FP, None), (F32, FP)])
def test_steps(lens, bits, grad, copy):
    c = Case(lens, bits, grad, copy)
    for k in range(4):
        c.step(seed=k)
        c.new_grads()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("grad,copy", [(BF, FP), (F32, None)])
def test_unaligned_tensors(bits, shift, grad, copy):
    c = Case([1000, 7, 260, 129], bits, grad, copy, shift)
    for _ in range(2):
        c.step()


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_as_they_are_packed(bits):
    """Gradients clipped into a flat buffer back to back, and parameters and copies in flat buffers."""
    lens = [1001, 3, 770, 64]
    c = Case(lens, bits, BF, BF)
    packed = torch.zeros(sum(lens) + 90, dtype=BF, device="cuda")
    Z.clip_gradients(c.grads, packed, max_norm=0.05)
    starts = np.cumsum([0] + lens)
    c.grads = [packed[a:a + n] for a, n in zip(starts, lens)]
    buffer = torch.randn(c.offsets[-1], device="cuda") * 0.1
    c.params = [buffer[o:o + n] for o, n in zip(c.offsets, lens)]
    c.step()
    c.step()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [64, 65, 640, 641, 1400])
def test_many_tensors(bits, n):
    """More tensors than a launch's table holds; some empty ones, at the ends too."""
    gen = torch.Generator().manual_seed(n)
    lens = (torch.rand(n, generator=gen) * 300).int().tolist()
    lens[0] = lens[-1] = lens[n // 2] = 0
    c = Case(lens, bits, BF, BF)
    for _ in range(3):
        c.step()


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_but_empty_tensors(bits):
    p = torch.empty(0, device="cuda")
    state = Z.adamw_state([p], bits)
    Z.adamw_step([p, p], [p, p], state, 1e-3)
    assert int(state.record[0]) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_coefficient_scale_and_skip(bits):
    c = Case([1000, 300], bits, FP, FP, std=1.0)
    c.step(loss_scale=1024.0, coef=torch.tensor([0.3], device="cuda"))
    c.step(loss_scale=3.0, coef=torch.tensor(0.7, device="cuda"), skip=torch.zeros(1, dtype=torch.int32, device="cuda"))
    kept = [t.clone() for t in (*c.params, *c.copies, *(t for t in c.state if t is not None))]
    Z.adamw_step(c.params, c.grads, c.state, 1e-3, copies=c.copies, skip=torch.ones((), dtype=torch.int32, device="cuda"))
    for a, b in zip(kept, (*c.params, *c.copies, *(t for t in c.state if t is not None))):
        assert torch.equal(a, b)
    c.step()


def test_with_the_norm_of_the_gradients():
    """gradient_norm's coefficient and flag, on the device, as clip_gradients gives them; an infinity skips the step."""
    c = Case([1000, 300, 77], 32, BF, None, std=1.0)
    norm, coef, bad = Z.gradient_norm(c.grads, max_norm=1.0)
    clipped = [g.clone() for g in c.grads]
    norm2, coef2, bad2 = Z.clip_gradients(clipped, max_norm=1.0)
    assert torch.equal(norm, norm2) and torch.equal(coef, coef2) and torch.equal(bad, bad2) and float(coef) < 0.1
    c.step(coef=coef, skip=bad)
    c.grads[1][5] = float("inf")
    norm, coef, bad = Z.gradient_norm(c.grads, max_norm=1.0)
    kept = [p.clone() for p in c.params]
    Z.adamw_step(c.params, c.grads, c.state, 1e-3, coef=coef, skip=bad)
    assert int(bad) == 1 and int(c.state.record[0]) == 1
    assert all(torch.equal(a, b) for a, b in zip(kept, c.params))


def test_the_bits_of_the_partitioned_step():
    """The same arithmetic as zero_adam_step, for constants that float holds exactly."""
    lens, steps = [4096 + 128], 5
    hp = dict(lr=2.0 ** -10, beta1=0.875, beta2=0.96875, eps=2.0 ** -27, weight_decay=0.125)
    plan = Z.ZeroPlan(-1, 1, lens, 128, 1, None, Z.ZERO_BF16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    master = torch.randn(plan.part_len, generator=gen, device="cuda")
    p = master.clone()
    m, v, g = (torch.zeros_like(p) for _ in range(3))
    param = torch.zeros(plan.psi_padded, dtype=BF, device="cuda")
    copy = torch.zeros_like(param)
    state = Z.adamw_state([p])
    for _ in range(steps):
        grad = torch.randn(plan.part_len, generator=gen, device="cuda").to(BF)
        plan.reduce(0, [grad], g, 1.0)
        plan.adam(0, g, master, m, v, param, hp["lr"], hp["beta1"], hp["beta2"], hp["eps"], hp["weight_decay"], 1, 1.0, 0.0)
        Z.adamw_step([p], [g], state, copies=[copy], **hp)
    plan.result()
    assert torch.equal(p, master) and torch.equal(state.m, m) and torch.equal(state.v, v) and torch.equal(copy, param)
    plan.close()


def test_moments_of_every_code():
    m = torch.arange(256, device="cuda", dtype=torch.int16).to(torch.uint8).view(torch.int8)
    m = torch.where(m.view(torch.uint8) % 128 == 127, torch.zeros_like(m), m)   # NaN codes are never written
    v = torch.arange(256, device="cuda", dtype=torch.int16).to(torch.uint8)
    scales = torch.tensor([0.37, 2.0 ** -100], device="cuda")
    state = Z.AdamWState(m, v, scales, scales, torch.zeros(2, dtype=torch.int64, device="cuda"))
    want_m, want_r, _, _ = values(state)
    for dtype in (F32, BF, FP):
        got_m, got_v = Z.adamw_moments(state, dtype)
        half = torch.finfo(dtype).eps / 2
        least = {F32: 2.0 ** -150, BF: 2.0 ** -134, FP: 2.0 ** -25}[dtype]
        assert ((got_m.double() - want_m).abs() <= half * want_m.abs() * (1 + 4 * U) + 2 * U * want_m.abs() + least).all()
        assert ((got_v.double() - want_r ** 2).abs() <= half * want_r ** 2 * (1 + 4 * U) + 4 * U * want_r ** 2 + least + 2.0 ** -149).all()
    full = Z.adamw_state([torch.zeros(300, device="cuda")])
    got = Z.adamw_moments(full, BF)
    assert got[0].dtype == BF and got[0].numel() == 384


def codes_of(x, top, bits, mantissa, low, most):
    """Codes and scales of float x >= 0 by torch's float operations, in the order that the definition gives."""
    rows = x.view(-1, BLOCK)
    scale = rows.amax(1, keepdim=True) * (1.0 / top)
    y = torch.where(scale > 0, rows * (1.0 / scale), 0.0).flatten()
    drop = 23 - mantissa
    z = y * 2.0 ** (-126 - low)       # float's subnormal numbers where the code has its
    code = (z.view(torch.int32) + (bits.int() << drop - 16) + (1 << drop - 17)) >> drop
    return code.clamp(max=most), scale.flatten()


@pytest.mark.parametrize("grad", [BF, F32])
def test_codes_to_the_bit(grad):
    """The definition's operations, each rounded on its own, give the kernel's codes and scales without an exception."""
    n = 1 << 21
    c = Case([n], 8, grad)
    coef = torch.tensor([0.37], device="cuda")
    for step in range(1, 5):
        c.new_grads()
        m0, r0, _, _ = (x.float() for x in values(c.state))
        f = c.grads[0].float() * (coef * torch.tensor(1 / 3.0, device="cuda"))
        m = m0 * 0.9 + f * (1 - 0.9)
        r = ((r0 * r0) * 0.999 + (f * f) * (1 - 0.999)).sqrt()
        c.step(check=False, seed=7, coef=coef, loss_scale=3.0)
        bits_m, bits_r = random16(0, n, step, 7)
        code_m, scale_m = codes_of(m.abs(), 448.0, bits_m, 3, -6, 126)
        code_r, scale_r = codes_of(r, 1.96875 / 256, bits_r, 5, -14, 255)
        _, _, got_m, got_r = values(c.state)
        assert torch.equal(c.state.m_scales, scale_m) and torch.equal(c.state.v_scales, scale_r)
        assert torch.equal(got_m, code_m.long()) and torch.equal(got_r, torch.where(r > 0, code_r.clamp(min=1), code_r).long())


def test_rounding_is_unbiased_and_depends_on_seed_step_and_place():
    """Means of codes over many elements of one value, to within five standard deviations."""
    n = 1 << 20
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), 0.3333, device="cuda")
    g[::BLOCK] = 1.0   # every block's largest
    seen = []
    for seed, steps in ((0, 1), (1, 1), (0, 2)):
        state = Z.adamw_state([p], 8)
        for _ in range(steps):
            Z.adamw_step([p], [g], state, 0.0, beta1=0.5, beta2=0.5, seed=seed)
        seen.append(state)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::BLOCK] = False
    for state in seen[:2]:
        m, r, _, _ = values(state)
        # m = g / 2, the root g sqrt(1/2), steps of 2^-3 and 2^-5 of their binade's start
        for got, want, step in ((m[rest], 0.5 * float(g[1]), 0.5 * 2.0 ** -2 / 8 * 448 / 448), (r[rest], math.sqrt(0.5) * float(g[1]), math.sqrt(0.5) * 2.0 ** -2 / 32 * 2)):
            assert len(got.unique()) == 2
            spread = float(got.max() - got.min())
            assert spread <= 2 * step
            deviation = spread / 2 / math.sqrt(got.numel())
            assert abs(float(got.mean()) - want) <= 5 * deviation + 2.0 ** -16 * spread + 8 * U * want
    # How often the second state has the first's code, if its own random bits know nothing of the first's: where the code
    # is the lower neighbour of the second's value, 1 - f of the time, where it is the upper one, f, with f the fraction
    # between them (a binomial mean, to five standard deviations).  A second step starts from the first's values.
    m1, r1, _, _ = values(seen[0])
    wide = g.double()
    for b, m, r in ((seen[1], 0.5 * wide, math.sqrt(0.5) * wide), (seen[2], 0.5 * m1 + 0.5 * wide, (0.5 * r1 ** 2 + 0.5 * wide ** 2).sqrt())):
        _, _, code_m, code_r = values(seen[0])
        _, _, other_m, other_r = values(b)
        for new, scale, code, other, places, low in ((m, b.m_scales, code_m, other_m, 3, -6), (r, b.v_scales, code_r, other_r, 5, -14)):
            y = new / scale.double().repeat_interleave(BLOCK)
            binade = torch.floor(torch.log2(y))
            place = y / torch.exp2(binade - places) + (binade - low) * 2 ** places
            f, under = place - place.floor(), place.floor().long()
            chance = torch.where(code == under, 1 - f, torch.where(code == under + 1, f, 0.0))[rest]
            same = (code == other).double()[rest]
            assert abs(float(same.mean() - chance.mean())) <= 5 * math.sqrt(float((chance * (1 - chance)).sum())) / chance.numel() + 2.0 ** -15
    # neighbours, and m against the root: independent to five standard deviations
    up_m = (seen[0].m.long() == seen[0].m[rest].long().max()).double()[rest]
    up_r = (seen[0].v.long() == seen[0].v[rest].long().max()).double()[rest]
    for x, y in ((up_m[1:], up_m[:-1]), (up_r[1:], up_r[:-1]), (up_m, up_r), (up_m[BLOCK:], up_m[:-BLOCK])):
        c = float(((x - x.mean()) * (y - y.mean())).mean() / (x.std() * y.std()))
        assert abs(c) <= 5 / math.sqrt(x.numel())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_block(value):
    c, d = Case([1000], 8, F32), Case([1000], 8, F32)
    d.grads[0][300] = value
    for _ in range(2):
        for x in (c, d):
            x.step(check=False)
    m, v = Z.adamw_moments(d.state)
    block = torch.zeros(1024, dtype=torch.bool, device="cuda")
    block[256:384] = True
    assert torch.isnan(m[block]).all() and torch.isnan(v[block]).all()
    assert torch.equal(d.state.m[~block], c.state.m[~block]) and torch.equal(d.state.v[~block], c.state.v[~block])
    assert torch.equal(d.params[0][384:], c.params[0][384:]) and torch.equal(d.params[0][:256], c.params[0][:256])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-18, 1e-12, 1e12, 1e18])
def test_sizes_of_gradients(bits, size):
    c = Case([700], bits, F32)
    for _ in range(3):
        c.grads[0].normal_(generator=c.gen).mul_(size)
        c.step(check=bits == 32 or size in (0.0, 1e-12, 1e12))
        assert torch.isfinite(c.params[0]).all()
    m, v = Z.adamw_moments(c.state)
    assert torch.isfinite(m).all() and (v >= 0).all()


def test_a_root_never_becomes_zero():
    """Elements far below their block's largest keep a root, so their update stays small."""
    p = torch.zeros(256, device="cuda")
    g = torch.full((256,), 1e-7, device="cuda")
    g[0] = 1.0
    state = Z.adamw_state([p], 8)
    for _ in range(50):
        Z.adamw_step([p], [g], state, 1e-3)
    assert (state.v[:128] >= 1).all()
    assert float(p.abs().max()) <= 50 * 1e-3 * 1.6


@pytest.mark.parametrize("bits", [32, 8])
def test_streams_graphs_and_repeats(bits):
    """The same bits on another stream; a captured step counts on with every replay; two graphs of two states at once."""
    def fresh(key):
        return Case([5000, 129, 1, 70000], bits, BF, BF, key=key)
    want = [fresh(k) for k in (1, 2)]
    for c in want:
        for _ in range(6):
            c.step(check=False)
    side = torch.cuda.Stream()
    other = fresh(1)
    torch.cuda.synchronize()
    for _ in range(6):
        Z.adamw_step(other.params, other.grads, other.state, copies=other.copies, stream=side, **HYPER)
    side.synchronize()
    cases, graphs, streams = [fresh(1), fresh(2)], [], [torch.cuda.Stream() for _ in range(2)]
    for c, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            Z.adamw_step(c.params, c.grads, c.state, copies=c.copies, **HYPER)
        graphs.append(g)
    for _ in range(6):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in ((other, want[0]), (cases[0], want[0]), (cases[1], want[1])):
        assert int(got.state.record[0]) == 6
        for a, b in zip((*got.params, *got.copies, *got.state), (*ref.params, *ref.copies, *ref.state)):
            assert a is b is None or torch.equal(a, b)


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """A tensor of more than 2^32 elements: the last ones' places and random bits, behind a short tensor."""
    lens = [1000, 2 ** 32 + 1000]
    gen = torch.Generator(device="cuda").manual_seed(1)
    params = [torch.zeros(n, device="cuda") for n in lens]
    grads = [torch.zeros(n, device="cuda", dtype=BF) for n in lens]
    last = 5000
    params[1][-last:] = torch.randn(last, generator=gen, device="cuda") * 0.1
    grads[1][-last:] = (torch.randn(last, generator=gen, device="cuda") * 1e-2).to(BF)
    state = Z.adamw_state(params, 8)
    p0 = params[1][-last:].double()
    Z.adamw_step(params, grads, state, seed=3, **HYPER)
    assert int((params[1][:-last] != 0).sum()) == 0 and int((state.m[:-6000] != 0).sum()) == 0
    at = 1024 + lens[1] - last
    first = at // BLOCK * BLOCK
    end = state.m.numel()
    assert first > 2 ** 32 - 4000 and end > 2 ** 32
    g = torch.zeros(end - first, dtype=torch.float64, device="cuda")
    g[at - first:at - first + last] = grads[1][-last:].double()
    m, r = (1 - HYPER["beta1"]) * g, math.sqrt(1 - HYPER["beta2"]) * g.abs()
    bits_m, bits_r = random16(first, end - first, 1, 3)
    cut = Z.AdamWState(state.m[first:], state.v[first:], state.m_scales[first // BLOCK:], state.v_scales[first // BLOCK:], None)
    _, _, code_m, code_r = values(cut)
    check_codes(m.abs(), 8 * U * m.abs(), cut.m_scales, code_m, bits_m, 3, -6, 126, False)
    check_codes(r, 8 * U * r, cut.v_scales, code_r, bits_r, 5, -14, 255, True)
    want = p0 * (1 - HYPER["lr"] * HYPER["weight_decay"]) - HYPER["lr"] * grads[1][-last:].double() / (grads[1][-last:].double().abs() + HYPER["eps"])
    assert ((params[1][-last:].double() - want).abs() <= 4 * U * (p0.abs() + want.abs()) + 2.0 ** -18 * HYPER["lr"]).all()


def test_refuses():
    c = Case([300, 40], 8, BF, BF)
    p, g, s, k = c.params, c.grads, c.state, c.copies
    bad = [
        lambda: Z.adamw_state(p, 16), lambda: Z.adamw_step([], [], s, 1e-3), lambda: Z.adamw_step(p, g[:1], s, 1e-3),
        lambda: Z.adamw_step(p, g, s, 1e-3, copies=k[:1]), lambda: Z.adamw_step(p, [g[0], g[1][:39]], s, 1e-3),
        lambda: Z.adamw_step([x.half() for x in p], g, s, 1e-3), lambda: Z.adamw_step(p, [g[0], g[1].float()], s, 1e-3),
        lambda: Z.adamw_step(p, [x.double() for x in g], s, 1e-3), lambda: Z.adamw_step(p, g, s, 1e-3, copies=[x.float() for x in k]),
        lambda: Z.adamw_step([p[0], p[0][:40]], g, s, 1e-3), lambda: Z.adamw_step([p[0], p[0]], [g[0], g[0]], s, 1e-3),
        lambda: Z.adamw_step(p, g, s._replace(m=s.m[:-128]), 1e-3), lambda: Z.adamw_step(p, g, s._replace(v=s.v.float()), 1e-3),
        lambda: Z.adamw_step(p, g, s._replace(m_scales=None), 1e-3), lambda: Z.adamw_step(p, g, s._replace(record=s.record.int()), 1e-3),
        lambda: Z.adamw_step(p, g, s, float("nan")), lambda: Z.adamw_step(p, g, s, 1e-3, beta1=1.0),
        lambda: Z.adamw_step(p, g, s, 1e-3, beta2=-0.1), lambda: Z.adamw_step(p, g, s, 1e-3, eps=-1.0),
        lambda: Z.adamw_step(p, g, s, 1e-3, loss_scale=0.0), lambda: Z.adamw_step(p, g, s, 1e-3, seed=2 ** 31),
        lambda: Z.adamw_step(p, g, s, 1e-3, coef=torch.ones(2, device="cuda")), lambda: Z.adamw_step(p, g, s, 1e-3, coef=torch.ones(1)),
        lambda: Z.adamw_step(p, g, s, 1e-3, skip=torch.ones(1, device="cuda")), lambda: Z.adamw_step([x.cpu() for x in p], g, s, 1e-3),
        lambda: Z.adamw_step([p[0].view(20, 15).t(), p[1]], [g[0].view(20, 15).t(), g[1]], s, 1e-3),
        lambda: Z.adamw_moments(s, torch.float64), lambda: Z.adamw_moments(s._replace(m=s.m[:-1])), lambda: Z.gradient_norm([]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(Z.ZeroError):
            call()
            print("not refused:", i)
    assert int(s.record[0]) == 0
    grown = [torch.nn.Parameter(x.clone()) for x in p]
    Z.adamw_step(grown, g, s, 1e-3)      # parameters that require grad are what an optimizer steps
    assert int(s.record[0]) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_what_an_iterator_gives(bits):
    """Tensors that nobody else holds, the same step as of a list of them."""
    a, b = Case([300, 40, 5000], bits, BF, BF), Case([300, 40, 5000], bits, BF, BF)
    for x, y in zip(a.params + a.grads, b.params + b.grads):
        y.copy_(x)
    Z.adamw_step(a.params, [g.float() for g in a.grads], a.state, 1e-3, copies=a.copies)
    Z.adamw_step((p.view(-1) for p in b.params), (g.float() for g in b.grads), b.state, 1e-3, copies=tuple(b.copies))
    for x, y in zip(a.params + a.copies, b.params + b.copies):
        assert torch.equal(x, y)
    for x, y in zip(a.state, b.state):
        assert x is None or torch.equal(x, y)


def test_the_smallest_eps():
    """2^-126 with moments of 0: the elements only decay."""
    p = [torch.full((300,), 2.0, device="cuda")]
    for bits in (32, 8):
        Z.adamw_step(p, [torch.zeros(300, device="cuda")], Z.adamw_state(p, bits), 1e-2, eps=2.0 ** -126, weight_decay=0.5)
    decay = torch.tensor(1 - 1e-2 * 0.5, dtype=torch.float64).float()
    assert (p[0].cpu() == decay * (decay * 2.0)).all()
