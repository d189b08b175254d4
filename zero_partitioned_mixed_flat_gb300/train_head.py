"""A small model trained end to end with the training head and the ZeRO step:

    python -m zero_partitioned_mixed_flat_gb300.train_head [--steps 60] [--ranks 2] [--wide 0] [--moments 32|8]

The model predicts a token from the two before it: the embedding of the last one
is added to a second embedding of the one before (the residual addition), the sum
is normalised, and the vocabulary matrix gives the logits.  A step is what a
training program does around the library:

    residual_norm -> linear_loss -> linear_loss_backward -> residual_norm_backward
    -> clip_gradients into a flat buffer per rank -> reduce, decision, AdamW, cast

Every rank (simulated on one GPU) takes its own batch; its four gradient tensors
are packed back to back into its flat buffer, as they are, and the flat buffers'
partitions are the slices that the reduce averages.  What is clipped is the average,
by the step's decision from the norm over all partitions: a rank's own norm says
nothing about it.  The model's weights are views of the parameter
buffer that the update writes.  Data is synthetic: the next token is the successor
of the last token or of the one before, with some noise, and some positions are
masked out of the loss.

--wide W puts a gated feed-forward block between: from the normalised sum, W gated
projections (gated_linear) and a product back, added to the sum, which is normalised again.
--moments 32 or 8 takes one rank's step over the list of weights instead of the ZeRO step: the
gradients' norm and flag stay on the device (gradient_norm), and adamw_step clips, updates
the float weights with moments of that many bits and rounds them into the model's.
"""
import argparse

import torch

from . import _abi as A
from .adamw import adamw_state, adamw_step
from .head import (check_losses, clip_gradients, gated_linear, gated_linear_backward, gradient_norm, linear_loss,
                   linear_loss_backward, residual_norm, residual_norm_backward)
from .plan import ZeroPlan
from .schedule import Hyper, StepBuffers, StepSchedule

EPS, IGNORE = 1e-5, -100


class BigramHead:
    """Weights as views of a flat buffer: two embeddings, the norm's weight, the vocabulary matrix; with a gated block
    its three matrices and the second norm's weight besides."""

    def __init__(self, vocab: int, dim: int, wide: int = 0):
        self.shapes = [(vocab, dim), (vocab, dim), (dim,), (vocab, dim)]
        self.stds = [0.5, 0.5, None, 0.05]
        if wide:
            self.shapes += [(wide, dim), (wide, dim), (dim, wide), (dim,)]
            self.stds += [dim ** -0.5, dim ** -0.5, 0.5 * wide ** -0.5, None]
        self.sizes = [torch.Size(s).numel() for s in self.shapes]

    def views(self, flat, offsets):
        return [flat[o:o + n].view(s) for o, n, s in zip(offsets, self.sizes, self.shapes)]

    def gradients(self, weights, tokens, targets, counted):
        """(mean loss over the counted tokens, gradients in the weights' order) of one batch."""
        last, before, scale, matrix, *block = weights
        first, total = residual_norm(last[tokens[:, 1]], before[tokens[:, 0]], scale, EPS)
        hidden = first
        if block:
            gate, up, down, second = block
            opened = gated_linear(first, gate, up)
            hidden, after = residual_norm(opened @ down.T, total, second, EPS)
        loss, lse = linear_loss(hidden, matrix, targets, ignore=IGNORE)
        upstream = torch.full_like(loss, 1.0 / counted)
        grad_hidden, grad_matrix = linear_loss_backward(hidden, matrix, targets, lse, upstream, ignore=IGNORE)
        grad_total, grad_block = None, []
        if block:
            grad_total, grad_second = residual_norm_backward(after, second, grad_hidden, None, EPS)
            grad_hidden, grad_gate, grad_up = gated_linear_backward(first, gate, up, grad_total @ down)
            grad_block = [grad_gate, grad_up, grad_total.T @ opened, grad_second]
        grad_sum, grad_scale = residual_norm_backward(total, scale, grad_hidden, grad_total, EPS)
        rows = grad_sum.float()
        grad_last, grad_before = (
            torch.zeros(matrix.shape, device=rows.device).index_add_(0, tokens[:, k], rows).to(matrix.dtype) for k in (1, 0))
        return loss.sum() / counted, [grad_last, grad_before, grad_scale, grad_matrix, *grad_block]


def start(model, weights, gen):
    for w, std in zip(weights, model.stds):
        w.copy_(torch.ones_like(w) if std is None else std * torch.randn(w.shape, generator=gen, device=w.device))


def batch(successors, n, gen):
    """n pairs of tokens, one of their two successors (a tenth random), and a tenth of the positions masked."""
    vocab, device = successors.shape[1], successors.device
    tokens = torch.randint(0, vocab, (n, 2), generator=gen, device=device)
    which = torch.randint(0, 2, (n, 1), generator=gen, device=device)
    targets = successors[which, tokens.gather(1, which)].squeeze(1)
    noise = torch.rand(n, generator=gen, device=device)
    targets = torch.where(noise < 0.1, torch.randint(0, vocab, (n,), generator=gen, device=device), targets)
    return tokens, torch.where(noise > 0.9, IGNORE, targets)


def train(steps=60, ranks=2, vocab=64, dim=128, tokens=2048, lr=2e-2, clip=1.0, seed=0, wide=0):
    """The losses of the steps, averaged over the ranks."""
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device).manual_seed(seed)
    model = BigramHead(vocab, dim, wide)
    plan = ZeroPlan(-1, ranks, model.sizes, 128, 2, None, A.ZERO_BF16)
    P, offsets = plan.part_len, plan.tensor_offsets
    params = torch.zeros(plan.psi_padded, dtype=torch.bfloat16, device=device)
    weights = model.views(params, offsets)
    start(model, weights, gen)
    master = {r: params[r * P:(r + 1) * P].float() for r in range(ranks)}
    moments = [{r: torch.zeros(P, device=device) for r in range(ranks)} for _ in range(2)]
    grads = {r: torch.empty(P, device=device) for r in range(ranks)}
    flats = torch.zeros(ranks, plan.psi_padded, dtype=torch.bfloat16, device=device)
    slices = {r: [flats[j, r * P:(r + 1) * P] for j in range(ranks)] for r in range(ranks)}
    buffers = StepBuffers(ranks=list(range(ranks)), slices=slices, g=grads, master=master, m=moments[0], v=moments[1],
                          param=params)
    step = StepSchedule(plan, buffers, Hyper(lr, 0.9, 0.99, 1e-8, 0.0, 1, clip), loss_scale=1.0)
    successors = torch.stack([torch.randperm(vocab, generator=gen, device=device) for _ in range(2)])
    losses = []
    for _ in range(steps):
        total = 0.0
        for j in range(ranks):
            pairs, targets = batch(successors, tokens, gen)
            loss, each = model.gradients(weights, pairs, targets, max(1, int((targets != IGNORE).sum())))
            clip_gradients(each, flats[j], offsets)
            total = total + loss / ranks
        StepSchedule.run(step.calls(torch.cuda.current_stream()))
        losses.append(float(total))
    check_losses()
    plan.result()
    plan.close()
    return losses


def train_whole(steps=60, vocab=64, dim=128, tokens=2048, lr=2e-2, clip=1.0, seed=0, wide=0, bits=32):
    """The losses of one rank's steps over whole tensors, the moments in `bits`."""
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device).manual_seed(seed)
    model = BigramHead(vocab, dim, wide)
    weights = [torch.empty(s, dtype=torch.bfloat16, device=device) for s in model.shapes]
    start(model, weights, gen)
    master = [w.float() for w in weights]
    state = adamw_state(master, bits)
    successors = torch.stack([torch.randperm(vocab, generator=gen, device=device) for _ in range(2)])
    losses = []
    for _ in range(steps):
        pairs, targets = batch(successors, tokens, gen)
        loss, grads = model.gradients(weights, pairs, targets, max(1, int((targets != IGNORE).sum())))
        _, coef, nonfinite = gradient_norm(grads, clip)
        adamw_step(master, grads, state, lr, 0.9, 0.99, 1e-8, copies=weights, coef=coef, skip=nonfinite, seed=seed)
        losses.append(float(loss))
    check_losses()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, help="partitions of the ZeRO step (2)")
    ap.add_argument("--wide", type=int, default=0, help="width of a gated block (a multiple of 8; 0: none)")
    ap.add_argument("--moments", type=int, choices=(8, 32), help="AdamW over whole tensors with moments of so many bits")
    args = ap.parse_args()
    if args.moments and args.ranks not in (None, 1):
        ap.error("--moments takes one rank's step over whole tensors: no --ranks")
    if args.moments:
        losses = train_whole(args.steps, wide=args.wide, bits=args.moments)
    else:
        losses = train(args.steps, 2 if args.ranks is None else args.ranks, wide=args.wide)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %4d  loss %.4f" % (i, losses[i]))
    print("step %4d  loss %.4f" % (len(losses) - 1, losses[-1]))


if __name__ == "__main__":
    main()
