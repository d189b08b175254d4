"""The head of a training step on torch tensors: residual addition and RMS norm,
the softmax cross entropy against the vocabulary matrix, their gradients, and
the clipped, packed gradients (the zero_norm_*, zero_loss_* and zero_clip_* calls
of include/zero.h).

These functions only allocate outputs and scratch, read strides off the tensors
and marshal them; the arithmetic runs in libzero.  Matrices are 2-D float16 or
bfloat16 CUDA tensors whose rows are contiguous; row lengths and strides must be
multiples of 8 and pointers 16-byte aligned.  `stream` is the current stream, a
torch.cuda.Stream or a raw cudaStream_t; outputs and scratch are allocated for
that stream, so a caller on several streams orders its own tensors between
them and nothing else.  Wrong shapes, types or devices raise ZeroError
(ZERO_EINVAL) before any device work.
"""
import numpy as np
import torch

from . import _abi as A

_LP = {torch.float16: A.ZERO_FP16, torch.bfloat16: A.ZERO_BF16}
_CLIP = {**_LP, torch.float32: A.ZERO_FP32}
_STATUS = {}   # device index -> the int32 that every loss call of the process ORs into


def _refuse(where, why):
    raise A.ZeroError(A.ZERO_EINVAL, where, why)


class _On:
    """Allocations inside belong to `stream` (None: the current stream)."""

    def __init__(self, stream):
        if stream is not None and not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        self.ctx = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _matrix(where, name, t, like=None, shape=None):
    """(rows, columns, row stride) of a 2-D tensor with contiguous rows."""
    if t.dim() != 2 or t.dtype not in _LP or not t.is_cuda:
        _refuse(where, "%s must be a 2-D float16 or bfloat16 CUDA tensor" % name)
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        _refuse(where, "%s differs in type or device" % name)
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        _refuse(where, "%s is %d x %d, expected %d x %d" % (name, rows, cols, *shape))
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        _refuse(where, "%s: the elements of a row must be contiguous" % name)
    # the stride of a single row (or of none) says nothing
    return rows, cols, s0 if rows > 1 else -(-cols // 8) * 8


def _vector(where, name, t, n, dtype, device):
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype or t.device != device or (n > 1 and t.stride(0) != 1):
        _refuse(where, "%s must be a contiguous vector of %d %s on %s" % (name, n, dtype, device))


def _status(device):
    word = _STATUS.get(device.index)
    if word is None:
        word = _STATUS[device.index] = torch.zeros(4, dtype=torch.int32, device=device)
        torch.cuda.synchronize(device)   # calls on any stream may use it from here on
    return word


def check_losses(device=None):
    """Waits for the device and raises if a linear_loss or linear_loss_backward
    since the last check met a target outside the vocabulary (ZERO_EINVAL) or
    gave up a bounded wait (ZERO_ETIMEOUT: its outputs are not valid)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    torch.cuda.synchronize(device)
    word = _status(device)
    bits = int(word[0].item())
    word.zero_()
    torch.cuda.synchronize(device)
    if bits & A.ZERO_LOSS_TIMEOUT:
        raise A.ZeroError(A.ZERO_ETIMEOUT, "check_losses", "a bounded device wait gave up")
    if bits & A.ZERO_LOSS_BAD_TARGET:
        raise A.ZeroError(A.ZERO_EINVAL, "check_losses", "a target lies outside the vocabulary")


# ---- residual addition + RMS norm ---------------------------------------------

def _norm_inputs(where, x, residual, weight):
    rows, dim, xs = _matrix(where, "x", x)
    rs = 0 if residual is None else _matrix(where, "residual", residual, x, (rows, dim))[2]
    _vector(where, "weight", weight, dim, x.dtype, x.device)
    return rows, dim, xs, rs


def residual_norm(x, residual, weight, eps, stream=None):
    """(out, sum): sum = x + residual (residual None: x), out = sum * rstd * weight
    with rstd = (mean(sum^2) + eps)^(-1/2) over each row."""
    rows, dim, xs, rs = _norm_inputs("residual_norm", x, residual, weight)
    with _On(stream):
        out = torch.empty((rows, dim), dtype=x.dtype, device=x.device)
        total = torch.empty((rows, dim), dtype=x.dtype, device=x.device)
        A.zero_norm_forward(x, xs, residual, rs, weight, eps, rows, dim, _LP[x.dtype], out, dim, total, dim,
                            stream)
    return out, total


def residual_norm_quantized(x, residual, weight, eps, fmt=A.ZERO_QUANT_INT8, stream=None):
    """(codes, scales, sum): residual_norm's out as int8 or E4M3 codes (one byte
    each, int8 tensor) with a float scale per block of 128 elements of a row."""
    rows, dim, xs, rs = _norm_inputs("residual_norm_quantized", x, residual, weight)
    with _On(stream):
        codes = torch.empty((rows, dim), dtype=torch.int8, device=x.device)
        scales = torch.empty((rows, -(-dim // A.ZERO_QUANT_BLOCK)), dtype=torch.float32, device=x.device)
        total = torch.empty((rows, dim), dtype=x.dtype, device=x.device)
        A.zero_norm_forward_quantized(x, xs, residual, rs, weight, eps, rows, dim, _LP[x.dtype], fmt, codes,
                                      scales, total, dim, stream)
    return codes, scales, total


def dequantize_rows(codes, scales, fmt, dtype, stream=None):
    """code * scale of its block, in `dtype`, for residual_norm_quantized's outputs."""
    where = "dequantize_rows"
    if codes.dim() != 2 or codes.dtype != torch.int8 or not codes.is_cuda or not codes.is_contiguous():
        _refuse(where, "codes must be a contiguous 2-D int8 CUDA tensor")
    rows, dim = codes.shape
    if (dtype not in _LP or scales.dtype != torch.float32 or scales.device != codes.device
            or scales.shape != (rows, -(-dim // A.ZERO_QUANT_BLOCK)) or not scales.is_contiguous()):
        _refuse(where, "scales must be one float32 per block of a row, dtype float16 or bfloat16")
    with _On(stream):
        out = torch.empty((rows, dim), dtype=dtype, device=codes.device)
        A.zero_dequantize_rows(codes, scales, fmt, rows, dim, _LP[dtype], out, dim, stream)
    return out


def residual_norm_backward(total, weight, grad_out, grad_sum, eps, stream=None):
    """(grad_in, grad_weight) of residual_norm: total is its second output, grad_out
    the gradient of its first, grad_sum (or None) what reaches the sum by its
    other uses.  grad_in is the gradient of x and of residual alike."""
    where = "residual_norm_backward"
    rows, dim, ts = _matrix(where, "total", total)
    _vector(where, "weight", weight, dim, total.dtype, total.device)
    gs = _matrix(where, "grad_out", grad_out, total, (rows, dim))[2]
    ss = 0 if grad_sum is None else _matrix(where, "grad_sum", grad_sum, total, (rows, dim))[2]
    with _On(stream):
        grad_in = torch.empty((rows, dim), dtype=total.dtype, device=total.device)
        grad_weight = torch.empty(dim, dtype=total.dtype, device=total.device)
        need = A.zero_norm_backward_workspace(rows, dim)
        space = torch.empty(need, dtype=torch.uint8, device=total.device)
        A.zero_norm_backward(total, ts, weight, grad_out, gs, grad_sum, ss, eps, rows, dim, _LP[total.dtype],
                             grad_in, dim, grad_weight, space, need, stream)
    return grad_in, grad_weight


# ---- cross entropy against the vocabulary matrix --------------------------------

def _loss_inputs(where, hidden, weight, targets):
    tokens, dim, hs = _matrix(where, "hidden", hidden)
    vocab, _, ws = _matrix(where, "weight", weight, hidden)
    if weight.shape[1] != dim:
        _refuse(where, "weight has rows of %d, hidden of %d" % (weight.shape[1], dim))
    _vector(where, "targets", targets, tokens, torch.int64, hidden.device)
    return tokens, dim, vocab, hs, ws


def linear_loss(hidden, weight, targets, ignore=-100, stream=None):
    """(loss, lse), float32 per token: the softmax cross entropy of hidden @ weight.T
    (weight: [vocab, dim]) against int64 targets, and the log-sum-exp the
    backward call takes.  The logits are never stored.  0 where a target is
    `ignore`; see check_losses for targets outside the vocabulary."""
    tokens, dim, vocab, hs, ws = _loss_inputs("linear_loss", hidden, weight, targets)
    with _On(stream):
        loss = torch.empty(tokens, dtype=torch.float32, device=hidden.device)
        lse = torch.empty(tokens, dtype=torch.float32, device=hidden.device)
        need = A.zero_loss_workspace(tokens, vocab, dim)[0]
        space = torch.empty(need, dtype=torch.uint8, device=hidden.device)
        A.zero_loss_forward(hidden, hs, weight, ws, targets, ignore, tokens, vocab, dim, _LP[hidden.dtype], loss,
                            lse, _status(hidden.device), space, need, stream)
    return loss, lse


def linear_loss_backward(hidden, weight, targets, lse, grad_loss, ignore=-100, grad_hidden=None,
                         grad_weight=None, stream=None):
    """(grad_hidden, grad_weight) of sum(grad_loss * loss), written into the given
    tensors if there are any (e.g. views of the flat gradient buffer)."""
    where = "linear_loss_backward"
    tokens, dim, vocab, hs, ws = _loss_inputs(where, hidden, weight, targets)
    _vector(where, "lse", lse, tokens, torch.float32, hidden.device)
    _vector(where, "grad_loss", grad_loss, tokens, torch.float32, hidden.device)
    with _On(stream):
        if grad_hidden is None:
            grad_hidden = torch.empty((tokens, dim), dtype=hidden.dtype, device=hidden.device)
        if grad_weight is None:
            grad_weight = torch.empty((vocab, dim), dtype=hidden.dtype, device=hidden.device)
        ghs = _matrix(where, "grad_hidden", grad_hidden, hidden, (tokens, dim))[2]
        gws = _matrix(where, "grad_weight", grad_weight, hidden, (vocab, dim))[2]
        need = A.zero_loss_workspace(tokens, vocab, dim)[1]
        space = torch.empty(need, dtype=torch.uint8, device=hidden.device)
        A.zero_loss_backward(hidden, hs, weight, ws, targets, ignore, tokens, vocab, dim, _LP[hidden.dtype], lse,
                             grad_loss, grad_hidden, ghs, grad_weight, gws, _status(hidden.device), space, need,
                             stream)
    return grad_hidden, grad_weight


# ---- global norm, clipping, packing ----------------------------------------------

def clip_gradients(grads, out=None, offsets=None, max_norm=0.0, loss_scale=1.0, stream=None):
    """(norm, coef, nonfinite), one-element device tensors: the global L2 norm of
    the contiguous gradient tensors `grads` (divided by loss_scale), the clipping
    coefficient, and whether an element is not finite.  The gradients times coef
    go to `out`: None writes them in place; a list takes one tensor each; a 1-D
    tensor is a flat buffer that takes them at `offsets` (elements; default: back
    to back, as ZeroPlan.tensor_offsets lays them out)."""
    where = "clip_gradients"
    if not grads:
        _refuse(where, "no gradients")
    dtype, device = grads[0].dtype, grads[0].device
    if dtype not in _CLIP or not grads[0].is_cuda:
        _refuse(where, "grads must be float16, bfloat16 or float32 CUDA tensors")
    lens = np.array([g.numel() for g in grads], np.int64)
    for g in grads:
        if g.dtype != dtype or g.device != device or not g.is_contiguous():
            _refuse(where, "grads must be contiguous, of one type and on one device")
    src = np.array([g.data_ptr() for g in grads], np.uint64)
    if out is None:
        dst = src
    elif isinstance(out, torch.Tensor):
        if out.dim() != 1 or out.dtype != dtype or out.device != device or not out.is_contiguous():
            _refuse(where, "out must be a contiguous 1-D tensor of the gradients' type and device")
        at = np.cumsum(lens) - lens if offsets is None else np.ascontiguousarray(offsets, np.int64)
        if at.shape != lens.shape or (at < 0).any() or (at + lens > out.numel()).any():
            _refuse(where, "a gradient does not fit into out at its offset")
        dst = at.astype(np.uint64) * np.uint64(out.element_size()) + np.uint64(out.data_ptr())
    else:
        if len(out) != len(grads) or any(o.dtype != dtype or o.device != device or o.numel() != n
                                         or not o.is_contiguous() for o, n in zip(out, lens)):
            _refuse(where, "out must hold one contiguous tensor of the same length and type per gradient")
        dst = np.array([o.data_ptr() for o in out], np.uint64)
    with _On(stream):
        norm, coef = torch.empty((), dtype=torch.float32, device=device), torch.empty((), dtype=torch.float32, device=device)
        nonfinite = torch.empty((), dtype=torch.int32, device=device)
        need = A.zero_clip_workspace(lens)
        space = torch.empty(need, dtype=torch.uint8, device=device)
        A.zero_clip_gradients(src, lens, _CLIP[dtype], dst, loss_scale, max_norm, norm, coef, nonfinite, space, need,
                              stream)
    return norm, coef, nonfinite
