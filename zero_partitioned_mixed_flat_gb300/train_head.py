"""A small model trained end to end with the training head and the ZeRO step:

    python -m zero_partitioned_mixed_flat_gb300.train_head [--steps 60] [--ranks 2]

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
"""
import argparse

import torch

from . import _abi as A
from .head import check_losses, clip_gradients, linear_loss, linear_loss_backward, residual_norm, residual_norm_backward
from .plan import ZeroPlan
from .schedule import Hyper, StepBuffers, StepSchedule

EPS, IGNORE = 1e-5, -100


class BigramHead:
    """Weights as views of a flat buffer: two embeddings, the norm's weight, the vocabulary matrix."""

    def __init__(self, vocab: int, dim: int):
        self.shapes = [(vocab, dim), (vocab, dim), (dim,), (vocab, dim)]
        self.sizes = [torch.Size(s).numel() for s in self.shapes]

    def views(self, flat, offsets):
        return [flat[o:o + n].view(s) for o, n, s in zip(offsets, self.sizes, self.shapes)]

    def gradients(self, weights, tokens, targets, counted):
        """(mean loss over the counted tokens, gradients in the weights' order) of one batch."""
        last, before, scale, matrix = weights
        hidden, total = residual_norm(last[tokens[:, 1]], before[tokens[:, 0]], scale, EPS)
        loss, lse = linear_loss(hidden, matrix, targets, ignore=IGNORE)
        upstream = torch.full_like(loss, 1.0 / counted)
        grad_hidden, grad_matrix = linear_loss_backward(hidden, matrix, targets, lse, upstream, ignore=IGNORE)
        grad_sum, grad_scale = residual_norm_backward(total, scale, grad_hidden, None, EPS)
        rows = grad_sum.float()
        grad_last, grad_before = (
            torch.zeros(matrix.shape, device=rows.device).index_add_(0, tokens[:, k], rows).to(matrix.dtype) for k in (1, 0))
        return loss.sum() / counted, [grad_last, grad_before, grad_scale, grad_matrix]


def batch(successors, n, gen):
    """n pairs of tokens, one of their two successors (a tenth random), and a tenth of the positions masked."""
    vocab, device = successors.shape[1], successors.device
    tokens = torch.randint(0, vocab, (n, 2), generator=gen, device=device)
    which = torch.randint(0, 2, (n, 1), generator=gen, device=device)
    targets = successors[which, tokens.gather(1, which)].squeeze(1)
    noise = torch.rand(n, generator=gen, device=device)
    targets = torch.where(noise < 0.1, torch.randint(0, vocab, (n,), generator=gen, device=device), targets)
    return tokens, torch.where(noise > 0.9, IGNORE, targets)


def train(steps=60, ranks=2, vocab=64, dim=128, tokens=2048, lr=2e-2, clip=1.0, seed=0):
    """The losses of the steps, averaged over the ranks."""
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device).manual_seed(seed)
    model = BigramHead(vocab, dim)
    plan = ZeroPlan(-1, ranks, model.sizes, 128, 2, None, A.ZERO_BF16)
    P, offsets = plan.part_len, plan.tensor_offsets
    params = torch.zeros(plan.psi_padded, dtype=torch.bfloat16, device=device)
    weights = model.views(params, offsets)
    for w, std in zip(weights, (0.5, 0.5, None, 0.05)):
        w.copy_(torch.ones_like(w) if std is None else std * torch.randn(w.shape, generator=gen, device=device))
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


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=2)
    args = ap.parse_args()
    losses = train(args.steps, args.ranks)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %4d  loss %.4f" % (i, losses[i]))
    print("step %4d  loss %.4f" % (len(losses) - 1, losses[-1]))


if __name__ == "__main__":
    main()
