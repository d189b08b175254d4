"""The head of a training step, operator by operator: its cases, inputs, plain forms and exact values.

Three operators, as one step meets them on its way from the last layer to the optimizer:

  norm   residual addition and root-mean-square norm of the rows of a layer's output, forward (in 16 bits, or in
         8 bits with a scale for every block of 128) and backward
  loss   softmax cross entropy of hidden states against a vocabulary matrix, without keeping the logits:
         the losses alone, or with the gradients of the hidden states and of the matrix
  clip   the global norm over a list of gradient tensors, and the clipped gradients packed into the flat buffer

`own` chooses between the plain form (torch operations in 32 bits) and the package's kernels.
"""
import math

import torch

own = False

LP = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
IGNORE = -100
BLOCK = 128          # elements that share a scale in the 8-bit forms
QUANTUM = 8 * 128    # the flat buffer is padded to eight partitions of whole 128-element runs
LARGEST = 8.0 * 4096 * 50257 * 4096  # operations of the largest loss case (logits twice, and both gradients)


def gpt2_block(d):
    return [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d, 4 * d * d, d]


def gpt2_lens(d, layers, vocab=50257, context=1024):
    return [vocab * d, context * d] + gpt2_block(d) * layers + [d, d]


def lens_of(case):
    """The lengths of the gradient tensors of a clip case, in list order."""
    if case["list"] == "gpt2":
        return gpt2_lens(case["width"], case["layers"])
    if case["list"] == "block":
        return gpt2_block(case["width"])
    gen = torch.Generator().manual_seed(case["shape_seed"])
    spread = math.log(case["longest"])
    return [int(math.exp(spread * u)) | 1 for u in torch.rand(case["tensors"], generator=gen, dtype=torch.float64).tolist()]


def listed():
    return [
        # one token scored at the smallest model: the weight matrix is read once, and latency shows
        dict(name="loss-one-token", op="loss", mode="loss", tokens=1, dim=768, vocab=50257, lp="fp16", ignored=0.0, pad=0),
        # evaluation of a shifted batch (every sequence of 1024 gives 1023 predictions)
        dict(name="loss-eval", op="loss", mode="loss", tokens=8 * 1023, dim=1600, vocab=50257, lp="bf16", ignored=0.0, pad=0),
        # one training sequence of the smallest model, some positions masked out of the loss
        dict(name="loss-train-small", op="loss", mode="train", tokens=1023, dim=768, vocab=50257, lp="bf16", ignored=0.1, pad=0),
        # two sequences of the 1.5B model with loss scaling
        dict(name="loss-train-xl", op="loss", mode="train", tokens=2048, dim=1600, vocab=50257, lp="fp16", ignored=0.0, pad=0),
        # four sequences of the 7.5B model: bound by the matrix products
        dict(name="loss-train-7.5b", op="loss", mode="train", tokens=4096, dim=4096, vocab=50257, lp="fp16", ignored=0.02, pad=0),
        # one row: what a single new token pays
        dict(name="norm-one-token", op="norm", mode="forward", rows=1, dim=4096, lp="bf16", format="none", residual=True, pad=0),
        # a short batch at the smallest width, int8 codes (six blocks a row)
        dict(name="norm-int8-small", op="norm", mode="forward", rows=1023, dim=768, lp="fp16", format="int8", residual=True, pad=0),
        # a long batch at the 1.5B width, fp8 codes (the thirteenth block of a row is half full)
        dict(name="norm-fp8-xl", op="norm", mode="forward", rows=16384, dim=1600, lp="bf16", format="fp8", residual=True, pad=0),
        # forward and backward of a large batch at the 7.5B width
        dict(name="norm-train-7.5b", op="norm", mode="train", rows=8191, dim=4096, lp="fp16", format="none", residual=True, pad=0),
        # one transformer block's gradients in 32 bits: two launches' latency
        dict(name="clip-block", op="clip", list="block", width=256, lp="fp32", std=1e-3, scale=1.0, clip=0.1),
        # every gradient of the smallest model (148 tensors)
        dict(name="clip-gpt2-small", op="clip", list="gpt2", width=768, layers=12, lp="bf16", std=1e-3, scale=1.0, clip=1.0),
        # every gradient of the 1.5B model (580 tensors), scaled by the loss scale
        dict(name="clip-gpt2-xl", op="clip", list="gpt2", width=1600, layers=48, lp="fp16", std=1e-3, scale=1024.0, clip=1.0),
    ]


def log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "norm", "norm", "clip"])
    lp = rng.choice(["fp16", "bf16"])
    pad = rng.choice([0, 0, 8, 264])                 # rows that are parts of wider rows
    width = 8 * (2 * log_int(rng, 4, 255) + 1)       # 72 .. 4088: odd multiples of 8
    if op == "loss":
        mode = rng.choice(["loss", "train"])
        tokens, vocab = log_int(rng, 1, 8191) | 1, log_int(rng, 64, 65536) | 1
        while (8.0 if mode == "train" else 2.0) * tokens * vocab * width > LARGEST:
            tokens = (tokens // 2) | 1
        return dict(op=op, mode=mode, tokens=tokens, dim=width, vocab=vocab, lp=lp, ignored=rng.choice([0.0, 0.1, 0.5]), pad=pad)
    if op == "norm":
        mode = rng.choice(["forward", "forward", "train"])
        rows = log_int(rng, 1, 16383) | 1
        fmt = rng.choice(["none", "int8", "fp8"]) if mode == "forward" else "none"
        return dict(op=op, mode=mode, rows=rows, dim=width, lp=lp, format=fmt, residual=rng.random() < 0.8, pad=pad)
    tensors = log_int(rng, 1, 600)
    return dict(op=op, list="random", tensors=tensors, longest=log_int(rng, 64, 2 ** 24), shape_seed=rng.randrange(2 ** 31),
                lp=rng.choice(["fp16", "bf16", "fp32"]), std=rng.choice([1e-5, 1e-3]), scale=rng.choice([1.0, 1024.0]),
                clip=rng.choice([0.0, 0.01, 1.0]))


def rows_of(gen, rows, dim, pad, dtype, std):
    """[rows, dim] normal values, part of rows of dim + pad elements."""
    wide = torch.randn(rows, dim + pad, generator=gen, device="cuda") * std
    return wide.to(dtype)[:, :dim]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = LP[case["lp"]]
    state = dict(case=case)
    if case["op"] == "loss":
        tokens, dim, vocab = case["tokens"], case["dim"], case["vocab"]
        weight = rows_of(gen, vocab, dim, 0, dtype, 0.02)
        targets = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        hidden = torch.randn(tokens, dim + case["pad"], generator=gen, device="cuda")
        # a model that has learned something: each target's logit stands 0 to 15 above the others' mean
        above = 15.0 * torch.rand(tokens, 1, generator=gen, device="cuda")
        hidden[:, :dim] += above * weight[targets].float() / (0.02 ** 2 * dim)
        drop = torch.rand(tokens, generator=gen, device="cuda") < case["ignored"]
        targets = torch.where(drop, IGNORE, targets)
        # the mean's gradient, times the loss scale: one that has settled where fp16 gradients do not overflow
        counted = max(1, tokens - int(drop.sum()))
        slope = min(65536.0 / counted, 64.0) if case["lp"] == "fp16" else 1.0 / counted
        state.update(hidden=hidden.to(dtype)[:, :dim], weight=weight, targets=targets,
                     grad_loss=torch.full((tokens,), slope, device="cuda"))
    elif case["op"] == "norm":
        rows, dim, pad = case["rows"], case["dim"], case["pad"]
        state.update(x=rows_of(gen, rows, dim, pad, dtype, 0.5), weight=(1.0 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(dtype))
        state["residual"] = rows_of(gen, rows, dim, pad, dtype, 2.0) if case["residual"] else None
        if case["mode"] == "train":
            state.update(grad_out=rows_of(gen, rows, dim, pad, dtype, 1e-2), grad_sum=rows_of(gen, rows, dim, pad, dtype, 1e-2))
    else:
        lens = lens_of(case)
        std = case["std"] * case["scale"]
        state["grads"] = [(torch.randn(n, generator=gen, device="cuda") * std).to(dtype) for n in lens]
        state["flat"] = torch.zeros(-(-sum(lens) // QUANTUM) * QUANTUM, dtype=dtype, device="cuda")
    return state


def run(state):
    case = state["case"]
    if own:
        return {"loss": own_loss, "norm": own_norm, "clip": own_clip}[case["op"]](case, state)
    return {"loss": plain_loss, "norm": plain_norm, "clip": plain_clip}[case["op"]](case, state)


def own_loss(case, s):
    import zero_partitioned_mixed_flat_gb300 as Z
    loss, lse = Z.linear_loss(s["hidden"], s["weight"], s["targets"], ignore=IGNORE)
    if case["mode"] == "loss":
        return {"loss": loss, "lse": lse}
    grad_hidden, grad_weight = Z.linear_loss_backward(s["hidden"], s["weight"], s["targets"], lse, s["grad_loss"], ignore=IGNORE)
    return {"loss": loss, "grad_hidden": grad_hidden, "grad_weight": grad_weight}


def own_norm(case, s):
    import zero_partitioned_mixed_flat_gb300 as Z
    if case["format"] != "none":
        fmt = Z.ZERO_QUANT_INT8 if case["format"] == "int8" else Z.ZERO_QUANT_FP8_E4M3
        codes, scales, total = Z.residual_norm_quantized(s["x"], s["residual"], s["weight"], EPS, fmt)
        return {"out": Z.dequantize_rows(codes, scales, fmt, s["x"].dtype), "scales": scales, "sum": total}
    out, total = Z.residual_norm(s["x"], s["residual"], s["weight"], EPS)
    if case["mode"] == "forward":
        return {"out": out, "sum": total}
    grad_in, grad_weight = Z.residual_norm_backward(total, s["weight"], s["grad_out"], s["grad_sum"], EPS)
    return {"out": out, "sum": total, "grad_in": grad_in, "grad_weight": grad_weight}


def own_clip(case, s):
    import zero_partitioned_mixed_flat_gb300 as Z
    norm, coef, nonfinite = Z.clip_gradients(s["grads"], s["flat"], max_norm=case["clip"], loss_scale=case["scale"])
    return {"flat": s["flat"], "norm": norm, "coef": coef, "nonfinite": nonfinite}


def loss_in(case, hidden, weight, targets, grad_loss, kind, lp):
    """The loss and its gradients with every sum in type `kind`; the gradients rounded to `lp` (None: not rounded)."""
    h, w = hidden.to(kind), weight.to(kind)
    logits = h @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top + (logits - top).exp().sum(1, keepdim=True).log()
    counts = targets != IGNORE
    at = torch.where(counts, targets, 0).unsqueeze(1)
    loss = torch.where(counts, (lse - logits.gather(1, at)).squeeze(1), 0.0)
    if case["mode"] == "loss":
        return {"loss": loss, "lse": lse.squeeze(1)}
    slope = logits.sub_(lse).exp_()
    slope.scatter_add_(1, at, torch.full_like(lse, -1.0))
    slope.mul_(torch.where(counts, grad_loss, 0.0).to(kind).unsqueeze(1))
    grad_hidden, grad_weight = slope @ w, slope.t() @ h
    return {"loss": loss, "grad_hidden": grad_hidden.to(lp or kind), "grad_weight": grad_weight.to(lp or kind)}


def plain_loss(case, s):
    return loss_in(case, s["hidden"], s["weight"], s["targets"], s["grad_loss"], torch.float32, s["hidden"].dtype)


def blocks_of(y):
    """[rows, blocks, BLOCK], the last block of a row filled up with zeros."""
    return torch.nn.functional.pad(y, (0, -y.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))


def plain_norm(case, s):
    lp = s["x"].dtype
    total = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    weight = s["weight"].float()
    rstd = torch.rsqrt(total.square().mean(1, keepdim=True) + EPS)
    out = total * rstd * weight
    if case["format"] != "none":
        y = blocks_of(out)
        top = y.abs().amax(2, keepdim=True)
        if case["format"] == "int8":
            scale = top / 127.0
            value = torch.where(scale > 0, (y / scale).round().clamp(-127, 127), 0.0) * scale
        else:
            scale = torch.ldexp(torch.ones_like(top), (torch.frexp(top).exponent - 8).clamp(-126, 120))
            scale = torch.where(top > 0, scale, 0.0)
            value = torch.where(scale > 0, (y / scale).to(torch.float8_e4m3fn).float(), 0.0) * scale
        return {"out": value.flatten(1)[:, :case["dim"]].to(lp), "scales": scale.squeeze(2), "sum": total.to(lp)}
    if case["mode"] == "forward":
        return {"out": out.to(lp), "sum": total.to(lp)}
    grad = s["grad_out"].float()
    along = (grad * weight * total).mean(1, keepdim=True) * rstd.square()
    grad_in = rstd * (grad * weight - total * along) + s["grad_sum"].float()
    grad_weight = (grad * total * rstd).sum(0)
    return {"out": out.to(lp), "sum": total.to(lp), "grad_in": grad_in.to(lp), "grad_weight": grad_weight.to(lp)}


def plain_clip(case, s):
    flat = torch.cat(s["grads"]).float()
    norm = flat.square().sum().sqrt() / case["scale"]
    coef = case["clip"] / (norm + 1e-6) if case["clip"] > 0 else torch.ones_like(norm)
    coef = torch.where(coef < 1, coef, 1.0)
    packed = torch.nn.functional.pad((flat * coef).to(s["flat"].dtype), (0, s["flat"].numel() - flat.numel()))
    return {"flat": packed, "norm": norm, "coef": coef, "nonfinite": (~torch.isfinite(flat)).any().to(torch.int32)}


def work(case):
    size = 4 if case["lp"] == "fp32" else 2
    if case["op"] == "loss":
        t, d, v = case["tokens"], case["dim"], case["vocab"]
        product = 2.0 * t * d * v
        inputs = size * (t * d + v * d) + 8 * t
        if case["mode"] == "loss":
            return {"bytes": inputs + 8 * t, "flops": product}
        # the least: the logits once and a product for each gradient
        return {"bytes": inputs + 4 * t + 4 * t + size * (t * d + v * d), "flops": 3 * product}
    if case["op"] == "norm":
        n, d = case["rows"] * case["dim"], case["dim"]
        read = n * size * (2 if case["residual"] else 1) + d * size
        if case["format"] != "none":
            return {"bytes": read + n + 4 * case["rows"] * -(-d // BLOCK) + n * size, "flops": 8.0 * n}
        if case["mode"] == "forward":
            return {"bytes": read + 2 * n * size, "flops": 6.0 * n}
        return {"bytes": read + 2 * n * size + 3 * n * size + d * size, "flops": 20.0 * n}
    n = sum(lens_of(case))
    return {"bytes": 2 * n * size + 12, "flops": 3.0 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "loss":
        if work(case)["flops"] > 6e12:
            return None
        return exact_loss(case, s)
    if case["op"] == "norm":
        return exact_norm(case, s)
    return exact_clip(case, s)


def exact_loss(case, s):
    hidden, weight, targets = s["hidden"].double(), s["weight"].double(), s["targets"]
    scores = torch.mm(hidden, weight.transpose(0, 1))
    lse = torch.logsumexp(scores, dim=1)
    row = torch.arange(case["tokens"], device=scores.device)[targets >= 0]
    loss = torch.zeros_like(lse)
    loss[row] = lse[row] - scores[row, targets[row]]
    if case["mode"] == "loss":
        return {"loss": loss, "lse": lse}
    chance = torch.softmax(scores, dim=1)
    chance[row, targets[row]] -= 1.0
    chance[targets < 0] = 0.0
    chance *= s["grad_loss"].double()[:, None]
    return {"loss": loss, "grad_hidden": torch.mm(chance, weight), "grad_weight": torch.mm(chance.transpose(0, 1), hidden)}


def exact_norm(case, s):
    total = s["x"].double()
    if s["residual"] is not None:
        total = total + s["residual"].double()
    weight, dim = s["weight"].double(), case["dim"]
    size = ((total ** 2).sum(dim=1) / dim + EPS) ** 0.5
    unit = total / size[:, None]
    out = unit * weight
    if case["format"] != "none":
        pieces = out.split(BLOCK, dim=1)
        tops = torch.stack([p.abs().max(dim=1).values for p in pieces], dim=1)
        if case["format"] == "int8":
            scales = tops / 127
            wide = scales.repeat_interleave(BLOCK, dim=1)[:, :dim]
            values = torch.round(out / wide) * wide
        else:
            scales = 2.0 ** (torch.floor(torch.log2(tops)) - 7).clamp(-126, 120)
            wide = scales.repeat_interleave(BLOCK, dim=1)[:, :dim]
            scaled = out / wide
            # E4M3: three bits below the leading one, and steps of 2^-9 below 2^-6
            step = 2.0 ** (torch.floor(torch.log2(scaled.abs().clamp_min(2.0 ** -6))) - 3)
            values = torch.round(scaled / step) * step * wide
        return {"out": values, "scales": scales, "sum": total}
    if case["mode"] == "forward":
        return {"out": out, "sum": total}
    grad = s["grad_out"].double()
    grad_unit = grad * weight
    grad_in = (grad_unit - unit * ((grad_unit * unit).sum(dim=1) / dim)[:, None]) / size[:, None] + s["grad_sum"].double()
    return {"out": out, "sum": total, "grad_in": grad_in, "grad_weight": (grad * unit).sum(dim=0)}


def exact_clip(case, s):
    norm = torch.stack([(g.double() ** 2).sum() for g in s["grads"]]).sum().sqrt() / case["scale"]
    coef = torch.ones_like(norm)
    if case["clip"] > 0:
        coef = torch.clamp(case["clip"] / (norm + 1e-6), max=1.0)
    packed = torch.zeros(s["flat"].numel(), dtype=torch.float64, device=norm.device)
    at = 0
    for g in s["grads"]:
        packed[at:at + g.numel()] = g.double() * coef
        at += g.numel()
    return {"flat": packed, "norm": norm, "coef": coef, "nonfinite": None}
