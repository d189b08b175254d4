"""A layer's gated projections and the optimizer's step over a list of tensors: cases, inputs, plain forms and exact values.

Two operators, next to the head of a training step (norm, loss, clipping) and before its update:

  gated  act(x gate^T) * (x up^T), the two projections, activation and product that open a gated feed-forward block:
         forward alone (from a single token to a long batch), or with the gradients of x and of both matrices
  adamw  one AdamW step over a list of parameter tensors with their gradients and 16-bit copies; the two moments are held
         in 32 bits, or in 8 bits with a scale for every block of 128

The 8-bit moments, for a tensor whose elements start at a multiple of 128 of the state: m as E4M3 codes times its block's
scale (the largest magnitude / 448); the square root of v as unsigned codes of three exponent and five mantissa bits,
which are the middle bits of a float16, times its block's scale (the largest / the largest code's value). Both are
rounded to one of the two neighbours by 16 random bits, a function of the seed, the step and the element's place.

`own` chooses between the plain form (torch operations in 32 bits) and the package's kernels.
"""
import math

import torch

own = False

LP = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128                          # elements of a moment that share a scale; tensors start at its multiples
TOP_M, TOP_R = 448.0, 1.96875 / 256  # the largest values of the two codes
LOW = 2.0 ** -126
M32 = 0xFFFFFFFF
HYPER = dict(lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.01)
LARGEST = 12.0 * 4096 * 4096 * 10928  # operations of the largest gated case


def gpt2_block(d):
    return [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d, 4 * d * d, d]


def lens_of(case):
    """The lengths of an adamw case's tensors, in list order."""
    if case["list"] == "gpt2":
        d = case["width"]
        return [50257 * d, 1024 * d] + gpt2_block(d) * case["layers"] + [d, d]
    if case["list"] == "block":
        return gpt2_block(case["width"])
    if case["list"] == "flat":
        return [case["longest"]]
    gen = torch.Generator().manual_seed(case["shape_seed"])
    spread = math.log(case["longest"])
    return [int(math.exp(spread * u)) | 1 for u in torch.rand(case["tensors"], generator=gen, dtype=torch.float64).tolist()]


def listed():
    return [
        # one new token at the smallest model's width: latency
        dict(name="gated-one-token-small", op="gated", mode="forward", tokens=1, dim=768, wide=2048, lp="fp16", act="silu", pad=0, masked=0.0),
        # one new token at the 7.5B model's width: both matrices are read once
        dict(name="gated-one-token-7.5b", op="gated", mode="forward", tokens=1, dim=4096, wide=10928, lp="bf16", act="silu", pad=0, masked=0.0),
        # a new token each of 48 sequences at the 1.5B model's width
        dict(name="gated-48-tokens", op="gated", mode="forward", tokens=48, dim=1600, wide=4264, lp="bf16", act="gelu_tanh", pad=0, masked=0.0),
        # evaluation of a batch of eight sequences at the 1.5B model's width
        dict(name="gated-eval-xl", op="gated", mode="forward", tokens=8 * 1023, dim=1600, wide=4264, lp="bf16", act="gelu", pad=0, masked=0.0),
        # one training sequence of the smallest model, some positions without a gradient
        dict(name="gated-train-small", op="gated", mode="train", tokens=1023, dim=768, wide=2048, lp="bf16", act="silu", pad=0, masked=0.1),
        # two sequences of the 1.5B model in fp16, its gradients scaled
        dict(name="gated-train-xl", op="gated", mode="train", tokens=2048, dim=1600, wide=4264, lp="fp16", act="gelu_tanh", pad=0, masked=0.0),
        # four sequences of the 7.5B model: bound by the matrix products
        dict(name="gated-train-7.5b", op="gated", mode="train", tokens=4096, dim=4096, wide=10928, lp="bf16", act="silu", pad=0, masked=0.0),
        # one transformer block's tensors, all in 32 bits: latency
        dict(name="adamw-block", op="adamw", bits=32, list="block", width=256, grad="fp32", copies="none", packed=False, skip=False),
        # every tensor of the smallest model, 32-bit moments, gradients packed back to back in a flat buffer
        dict(name="adamw-gpt2-small", op="adamw", bits=32, list="gpt2", width=768, layers=12, grad="bf16", copies="bf16", packed=True, skip=False),
        # the same with 8-bit moments and gradients as they come from a backward pass
        dict(name="adamw8-gpt2-small", op="adamw", bits=8, list="gpt2", width=768, layers=12, grad="bf16", copies="bf16", packed=False, skip=False),
        # a rank's partition of the 7.5B model over 64 ranks, as one tensor with the reduced float gradient
        dict(name="adamw-partition", op="adamw", bits=32, list="flat", longest=117189632, grad="fp32", copies="fp16", packed=False, skip=False),
        # every tensor of the 1.5B model, 8-bit moments
        dict(name="adamw8-gpt2-xl", op="adamw", bits=8, list="gpt2", width=1600, layers=48, grad="fp16", copies="fp16", packed=False, skip=False),
    ]


def log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    if rng.random() < 0.6:
        lp, act, mode = rng.choice(["fp16", "bf16"]), rng.choice(["silu", "gelu", "gelu_tanh"]), rng.choice(["forward", "train"])
        dim = 8 * (2 * log_int(rng, 4, 255) + 1)    # 72 .. 4088: odd multiples of 8
        wide = 8 * (2 * log_int(rng, 8, 682) + 1)   # 136 .. 10920
        tokens = log_int(rng, 1, 8191) | 1
        while (12.0 if mode == "train" else 4.0) * tokens * dim * wide > LARGEST:
            tokens = tokens // 2 | 1
        return dict(op="gated", mode=mode, tokens=tokens, dim=dim, wide=wide, lp=lp, act=act, pad=rng.choice([0, 0, 8, 264]), masked=rng.choice([0.0, 0.3]))
    case = dict(op="adamw", bits=rng.choice([8, 32]), grad=rng.choice(["fp16", "bf16", "fp32"]), copies=rng.choice(["none", "fp16", "bf16"]),
                packed=rng.choice([False, True]), skip=rng.random() < 0.1, list=rng.choice(["gpt2", "random", "random"]))
    if case["list"] == "gpt2":
        return dict(case, width=64 * rng.randint(2, 12), layers=rng.randint(2, 12))
    return dict(case, tensors=rng.randint(1, 700), longest=log_int(rng, 1000, 10_000_000), shape_seed=rng.randrange(1 << 30))


def rows_of(gen, rows, dim, pad, dtype, std):
    """[rows, dim] normal values, part of rows of dim + pad elements."""
    wide = torch.randn(rows, dim + pad, generator=gen, device="cuda") * std
    return wide.to(dtype)[:, :dim]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (prepare_gated if case["op"] == "gated" else prepare_adamw)(case, gen, seed)


def prepare_gated(case, gen, seed):
    dtype, tokens, dim, wide = LP[case["lp"]], case["tokens"], case["dim"], case["wide"]
    state = dict(case=case, x=rows_of(gen, tokens, dim, case["pad"], dtype, 1.0),
                 gate=rows_of(gen, wide, dim, 0, dtype, 0.02), up=rows_of(gen, wide, dim, 0, dtype, 0.02))
    if case["mode"] == "train":
        grad = torch.randn(tokens, wide + case["pad"], generator=gen, device="cuda") * (1e-2 if case["lp"] == "fp16" else 1e-4)
        grad[torch.rand(tokens, generator=gen, device="cuda") < case["masked"]] = 0.0
        state["grad"] = grad.to(dtype)[:, :wide]
    return state


def prepare_adamw(case, gen, seed):
    lens = lens_of(case)
    starts, total = [], 0
    for n in lens:
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    master = torch.randn(total, generator=gen, device="cuda").mul_(0.02)
    inside = torch.ones(total, dtype=torch.bool, device="cuda")
    for n, o in zip(lens, starts):
        inside[o + n:o + -(-n // BLOCK) * BLOCK] = False
    master.mul_(inside)
    lp = LP.get(case["copies"])
    copy = master.to(lp) if lp else None
    views = lambda flat: [flat[o:o + n] for n, o in zip(lens, starts)]  # noqa: E731
    # gradients of a step: each tensor has a size of its own
    kind = LP[case["grad"]]
    sizes = torch.exp(torch.randn(len(lens), generator=gen, device="cuda")).mul_(1e-3 if kind != torch.float16 else 1e-2).tolist()
    if case["packed"]:
        flat = torch.randn(sum(lens), generator=gen, device="cuda")
        grads = list(flat.split(lens))
        for g, size in zip(grads, sizes):
            g.mul_(size)
        grads = list(flat.to(kind).split(lens))
    else:
        grads = [torch.randn(n, generator=gen, device="cuda").mul_(size).to(kind) for n, size in zip(lens, sizes)]
    # moments as some steps have left them
    if case["bits"] == 32:
        m = torch.randn(total, generator=gen, device="cuda").mul_(2e-4).mul_(inside)
        v = torch.randn(total, generator=gen, device="cuda").mul_(1e-3).square_().mul_(inside)
        moments = (m, v, None, None)
    else:
        m = torch.randn(total, generator=gen, device="cuda").mul_(100.0).clamp_(-TOP_M, TOP_M).mul_(inside).to(torch.float8_e4m3fn).view(torch.int8)
        r = torch.randint(40, 256, (total,), dtype=torch.uint8, generator=gen, device="cuda").mul_(inside)
        scales = [torch.rand(total // BLOCK, generator=gen, device="cuda").add_(0.5).mul_(top) for top in (1e-3 / TOP_M, 3e-3 / TOP_R)]
        moments = (m, r, *scales)
    record = torch.tensor([10 + seed % 500, 0], dtype=torch.int64, device="cuda")
    return dict(case=case, lens=lens, master=master, params=views(master), copy=copy, copies=None if copy is None else views(copy),
                grads=grads, state=(*moments, record), seed=seed % 1000,
                loss_scale=1024.0 if kind == torch.float16 else 1.0,
                coef=torch.full((1,), 0.5 + 0.5 * (seed % 97) / 97, device="cuda"),
                nonfinite=torch.full((1,), int(case["skip"]), dtype=torch.int32, device="cuda"))


def run(state):
    case = state["case"]
    if own:
        return (own_gated if case["op"] == "gated" else own_adamw)(case, state)
    return (plain_gated if case["op"] == "gated" else plain_adamw)(case, state)


def own_gated(case, s):
    import zero_partitioned_mixed_flat_gb300 as Z
    out = Z.gated_linear(s["x"], s["gate"], s["up"], case["act"])
    if case["mode"] == "forward":
        return {"out": out}
    grad_x, grad_gate, grad_up = Z.gated_linear_backward(s["x"], s["gate"], s["up"], s["grad"], case["act"])
    return {"out": out, "grad_x": grad_x, "grad_gate": grad_gate, "grad_up": grad_up}


def own_adamw(case, s):
    import zero_partitioned_mixed_flat_gb300 as Z
    Z.adamw_step(s["params"], s["grads"], s["state"], HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], HYPER["wd"],
                 copies=s["copies"], loss_scale=s["loss_scale"], coef=s["coef"], skip=s["nonfinite"], seed=s["seed"])
    m, v = s["state"][:2]
    if case["bits"] == 8:
        m, v = Z.adamw_moments(s["state"], torch.bfloat16)
    return {"params": s["master"], "copies": s["copy"], "m": m, "v": v}


def act_and_slope(kind, a):
    """The activation and its derivative at a."""
    if kind == "silu":
        s = a.sigmoid()
        return a * s, s * (1.0 + a * (1.0 - s))
    if kind == "gelu_tanh":
        inner = math.sqrt(2.0 / math.pi) * (a + 0.044715 * a.pow(3))
        half = 0.5 * (1.0 + inner.tanh())
        return a * half, half + 0.5 * a * (1.0 - inner.tanh().square()) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * a.square())
    half = 0.5 * torch.erfc(a * -math.sqrt(0.5))
    return a * half, half + a * (a.square() * -0.5).exp() * (1.0 / math.sqrt(2.0 * math.pi))


def plain_gated(case, s):
    lp = s["x"].dtype
    x, gate, up = s["x"].float(), s["gate"].float(), s["up"].float()
    b = x @ up.t()
    act, slope = act_and_slope(case["act"], x @ gate.t())
    out = (act * b).to(lp)
    if case["mode"] == "forward":
        return {"out": out}
    grad = s["grad"].float()
    grad_a, grad_b = grad * b * slope, grad * act
    return {"out": out, "grad_x": (grad_a @ gate + grad_b @ up).to(lp), "grad_gate": (grad_a.t() @ x).to(lp), "grad_up": (grad_b.t() @ x).to(lp)}


def mix(x):
    """Numbers below 2^32 to others, one to one."""
    x = x ^ x >> 16
    x = (x * 0x9E3779B1) & M32
    x = x ^ x >> 15
    x = (x * 0xB504F333) & M32
    return x ^ x >> 16


def random_bits(total, step, seed):
    """(16 bits for m, 16 bits for the root of v) of every element."""
    at = torch.arange(total, dtype=torch.int64, device=step.device)
    key = mix((mix(torch.full_like(step, seed)) + step) & M32)
    word = mix((at & M32) ^ mix((key + (at >> 32)) & M32))
    return (word & 0xFFFF).int(), (word >> 16).int()


def rounded(y, bits, mantissa, low):
    """Codes of y >= 0: the float's bits from the mantissa's last place on, 0 at 0, steps that are equal below `low` (a power of two), rounded by random bits."""
    drop = 23 - mantissa
    below = y < low
    first = torch.tensor(low).view(torch.int32).item() >> drop
    word = torch.where(below, y + low, y).view(torch.int32) + (bits << (drop - 16)) + (1 << (drop - 17))
    return (word >> drop) - torch.where(below, first, first - (1 << mantissa))


def encoded(x, top, bits, mantissa, low, most):
    """(codes, scales) of x >= 0."""
    rows = x.view(-1, BLOCK)
    scale = rows.amax(1, keepdim=True) * (1.0 / top)
    scale = torch.where(scale >= LOW, scale, 0.0)
    y = torch.where(scale > 0, rows * (1.0 / scale), 0.0).flatten()
    return rounded(y, bits, mantissa, low).clamp_(max=most), scale.flatten()


def values_m(codes, scales):
    return (codes.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * scales[:, None]).flatten()


def values_r(codes, scales):
    return ((codes.to(torch.int16) << 5).view(torch.float16).float().view(-1, BLOCK) * scales[:, None]).flatten()


def padded(tensors):
    """One flat float tensor, each part filled up with zeros to whole blocks."""
    zeros = torch.zeros(BLOCK, device=tensors[0].device, dtype=tensors[0].dtype)
    return torch.cat([x for t in tensors for x in (t, zeros[:-t.numel() % BLOCK])]).float()


def plain_adamw(case, s):
    m, v, m_scales, v_scales, record = s["state"]
    if case["bits"] == 8:
        m_old, v_old = values_m(m, m_scales), values_r(v, v_scales).square()
    else:
        m_old, v_old = m, v
    keep = s["nonfinite"] != 0
    step = record[:1] + 1
    bc1, bc2 = ((1.0 - HYPER[b] ** step.double()).float() for b in ("beta1", "beta2"))
    grad = padded(s["grads"]) * (s["coef"] / s["loss_scale"])
    m_new = m_old * HYPER["beta1"] + grad * (1.0 - HYPER["beta1"])
    v_new = v_old * HYPER["beta2"] + grad.square() * (1.0 - HYPER["beta2"])
    update = (m_new / bc1 * HYPER["lr"]) / ((v_new / bc2).sqrt() + HYPER["eps"])
    s["master"].copy_(torch.where(keep, s["master"], s["master"] * (1.0 - HYPER["lr"] * HYPER["wd"]) - update))
    del update, grad, m_old, v_old
    if s["copy"] is not None:
        s["copy"].copy_(torch.where(keep, s["copy"], s["master"].to(s["copy"].dtype)))
    if case["bits"] == 8:
        bits_m, bits_r = random_bits(m.numel(), step, s["seed"])
        codes, scales = encoded(m_new.abs(), TOP_M, bits_m, 3, 2.0 ** -6, 126)
        m.copy_(torch.where(keep, m, (codes + (m_new < 0) * 128).to(torch.uint8).view(torch.int8)))
        m_scales.copy_(torch.where(keep, m_scales, scales))
        root = v_new.sqrt_()
        codes, scales = encoded(root, TOP_R, bits_r, 5, 2.0 ** -14, 255)
        v.copy_(torch.where(keep, v, torch.where((root > 0) & (codes == 0), 1, codes).to(torch.uint8)))
        v_scales.copy_(torch.where(keep, v_scales, scales))
        m_out, v_out = values_m(m, m_scales).bfloat16(), values_r(v, v_scales).square().bfloat16()
    else:
        m_out, v_out = m.copy_(torch.where(keep, m, m_new)), v.copy_(torch.where(keep, v, v_new))
    record[:1].copy_(torch.where(keep, record[:1], step))
    return {"params": s["master"], "copies": s["copy"], "m": m_out, "v": v_out}


def work(case):
    if case["op"] == "gated":
        t, d, f = case["tokens"], case["dim"], case["wide"]
        product = 2.0 * t * d * f
        read = 2 * (t * d + 2 * f * d)
        if case["mode"] == "forward":
            return {"bytes": read + 2 * t * f, "flops": 2 * product}
        # both projections, and two products for the gradient of x and one for each matrix's
        return {"bytes": read + 2 * t * f + 2 * t * f + 2 * (t * d + 2 * f * d), "flops": 6 * product}
    n = sum(lens_of(case))
    grad, copy = {"fp32": 4, "none": 0}.get(case["grad"], 2), {"none": 0}.get(case["copies"], 2)
    # parameters and moments read and written; the 8-bit moments handed over in 16 bits besides
    moments = 16 if case["bits"] == 32 else 4 + 4 * 4 / BLOCK + 2 + 4
    return {"bytes": (8 + grad + copy + moments) * n, "flops": 16.0 * n}


def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return exact_gated(case, s) if case["op"] == "gated" else exact_adamw(case, s)


def exact_gated(case, s):
    x, gate, up = s["x"].double(), s["gate"].double(), s["up"].double()
    g, u = torch.mm(x, gate.transpose(0, 1)), torch.mm(x, up.transpose(0, 1))
    # each activation is g * p(g); dp is the derivative of p
    if case["act"] == "silu":
        p = 1 / (1 + torch.exp(-g))
        dp = p * (1 - p)
    elif case["act"] == "gelu":
        p = torch.special.ndtr(g)
        dp = torch.exp(-g * g / 2) / (2 * math.pi) ** 0.5
    else:
        c = (2 / math.pi) ** 0.5
        p = 1 / (1 + torch.exp(-2 * c * (g + 0.044715 * g ** 3)))
        dp = p * (1 - p) * 2 * c * (1 + 0.134145 * g ** 2)
    out = g * p * u
    if case["mode"] == "forward":
        return {"out": out}
    d = s["grad"].double()
    dg, du = d * u * (p + g * dp), d * g * p
    return {"out": out, "grad_x": torch.mm(dg, gate).addmm_(du, up), "grad_gate": torch.mm(dg.transpose(0, 1), x), "grad_up": torch.mm(du.transpose(0, 1), x)}


def exact_codes(y, bits, places, exponent):
    """The values of codes with `places` mantissa bits and normal from 2^exponent on, for y >= 0, and the code itself being 0."""
    step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** exponent))).clamp_min(exponent) - places)
    return torch.floor(y / step + (bits.double() + 0.5) / 65536) * step


def exact_adamw(case, s):
    """A stretch of whole blocks at a time: the longest lists have no room for all of it in 64 bits."""
    m, v, m_scales, v_scales, record = s["state"]
    master, total, eight = s["master"], s["master"].numel(), case["bits"] == 8
    grads = torch.zeros(total, dtype=s["grads"][0].dtype, device=master.device)
    at = 0
    for g in s["grads"]:
        grads[at:at + g.numel()] = g
        at += -(-g.numel() // BLOCK) * BLOCK
    t = int(record[0]) + 1
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    factor = float(s["coef"]) / s["loss_scale"]
    kept = torch.float64 if total < 1 << 28 else torch.float32
    out = {k: torch.empty(total, dtype=kept, device=master.device) for k in ("params", "m", "v")}
    for a in range(0, total, 1 << 26):
        z = min(total, a + (1 << 26))
        old_m, old_v, p = m[a:z], v[a:z], master[a:z].double()
        if eight:
            spread = lambda x: x[a // BLOCK:z // BLOCK].double().repeat_interleave(BLOCK)  # noqa: E731
            code = v[a:z].long()
            exponent, mantissa = code // 32, code % 32
            old_v = (torch.where(exponent > 0, (32 + mantissa) * torch.exp2(exponent.double() - 20), mantissa * 2.0 ** -19) * spread(v_scales)) ** 2
            code = m[a:z].view(torch.uint8).long()
            exponent, mantissa = code % 128 // 8, code % 8
            old_m = torch.where(exponent > 0, (8 + mantissa) * torch.exp2(exponent.double() - 10), mantissa * 2.0 ** -9) * spread(m_scales)
            old_m = torch.where(code > 127, -old_m, old_m)
        g = grads[a:z].double() * factor
        new_m, new_v = b1 * old_m.double() + (1 - b1) * g, b2 * old_v.double() + (1 - b2) * g ** 2
        if case["skip"]:
            new_m, new_v, new_p = old_m.double(), old_v.double(), p
        else:
            new_p = p - HYPER["lr"] * (HYPER["wd"] * p + (new_m / (1 - b1 ** t)) / ((new_v / (1 - b2 ** t)) ** 0.5 + HYPER["eps"]))
        out["params"][a:z] = new_p
        if eight and not case["skip"]:
            bits_m, bits_r = bits_between(a, z, t, s["seed"], master.device)
            for name, new, bits, top, places, exponent in (("m", new_m, bits_m, TOP_M, 3, -6), ("v", new_v ** 0.5, bits_r, TOP_R, 5, -14)):
                scale = new.abs().view(-1, BLOCK).amax(1, keepdim=True) / top
                scale = torch.where(scale >= LOW, scale, 0.0)
                y = torch.where(scale > 0, new.abs().view(-1, BLOCK) / scale, 0.0).flatten()
                value = exact_codes(y, bits, places, exponent).clamp_max(top)
                if name == "v":
                    value = torch.where((new > 0) & (value == 0), 2.0 ** -19, value)
                value = (value.view(-1, BLOCK) * scale).flatten()
                out[name][a:z] = value * new.sign() if name == "m" else value ** 2
        else:
            out["m"][a:z], out["v"][a:z] = new_m, new_v
    copies = None if s["copy"] is None else out["params"]
    return {"params": out["params"], "copies": copies, "m": out["m"], "v": out["v"]}


def bits_between(a, z, step, seed, device):
    """Elements [a, z)'s random bits: the low 16 of a number for m, the high 16 for the root of v."""
    def scramble(x):
        for shift, factor in ((16, 0x9E3779B1), (15, 0xB504F333), (16, 1)):
            x = ((x ^ (x >> shift)) * factor) % (1 << 32)
        return x
    key = scramble((scramble(seed) + step) % (1 << 32))
    place = torch.arange(a, z, dtype=torch.int64, device=device)
    high = torch.tensor([scramble((key + h) % (1 << 32)) for h in range((z >> 32) + 1)], dtype=torch.int64, device=device)
    word = scramble((place % (1 << 32)) ^ high[place >> 32])
    return word % 65536, word // 65536
