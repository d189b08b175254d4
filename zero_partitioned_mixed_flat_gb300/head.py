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
them and nothing else.  No graph is recorded: the *_backward functions are the
gradients, to be called by hand or from a torch.autograd.Function, and a matrix
or vector that requires grad is refused while gradients are enabled (clip_gradients
takes its tensors as numbers).  Wrong shapes, types or devices raise ZeroError
(ZERO_EINVAL) before any device work.  A process's first loss call on a device
allocates its status word and waits for the device, so it belongs before a graph
capture; everything else can be captured.
"""
import contextlib
import threading
from array import array
from ctypes import byref, c_int64 as _i64
from itertools import accumulate
from operator import attrgetter

import numpy as np
import torch

from . import _abi as A

_LP = {torch.float16: A.ZERO_FP16, torch.bfloat16: A.ZERO_BF16}
_CLIP = {**_LP, torch.float32: A.ZERO_FP32}
_STATUS = {}   # device index -> the int32 that every loss call of the process ORs into
_STATUS_LOCK = threading.Lock()
_HERE = contextlib.nullcontext()


def _refuse(where, why):
    raise A.ZeroError(A.ZERO_EINVAL, where, why)


def _call(name, *args):
    """One libzero call; args are numbers and addresses."""
    code = getattr(A.load(), name)(*args)
    if code:
        A._check(code, name)


def _on(stream):
    """A context whose allocations belong to `stream` (None: the current stream)."""
    if stream is None:
        return _HERE
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _addr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _scratch(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device)


def _plain(where, name, t):
    if t.requires_grad and torch.is_grad_enabled():
        _refuse(where, "%s requires grad, and the call would record no graph: detach it, or call under torch.no_grad()" % name)


def _matrix(where, name, t, dtype=None, shape=None):
    """(rows, columns, row stride) of a 2-D tensor with contiguous rows on the current device."""
    _plain(where, name, t)
    if t.ndim != 2 or t.dtype not in _LP or t.get_device() != torch._C._cuda_getDevice():
        _refuse(where, "%s must be a 2-D float16 or bfloat16 tensor on the current CUDA device" % name)
    if dtype is not None and t.dtype != dtype:
        _refuse(where, "%s is %s, expected %s" % (name, t.dtype, dtype))
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        _refuse(where, "%s is %d x %d, expected %d x %d" % (name, rows, cols, *shape))
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        _refuse(where, "%s: the elements of a row must be contiguous" % name)
    # the stride of a single row (or of none) says nothing
    return rows, cols, s0 if rows > 1 else -(-cols // 8) * 8


def _vector(where, name, t, n, dtype):
    _plain(where, name, t)
    if (t.ndim != 1 or t.dtype != dtype or t.get_device() != torch._C._cuda_getDevice() or t.shape[0] != n
            or (n > 1 and t.stride(0) != 1)):
        _refuse(where, "%s must be a contiguous vector of %d %s on the current CUDA device" % (name, n, dtype))


def _status(device):
    word = _STATUS.get(device.index)
    if word is None:
        with _STATUS_LOCK:               # one word, whichever thread calls first
            word = _STATUS.get(device.index)
            if word is None:
                word = torch.zeros(4, dtype=torch.int32, device=device)
                torch.cuda.synchronize(device)   # calls on any stream may use it from here on
                _STATUS[device.index] = word
    return word


def check_losses(device=None):
    """Waits for the device and raises if a linear_loss or linear_loss_backward
    since the last check met a target outside the vocabulary (ZERO_EINVAL) or
    gave up a bounded wait (ZERO_ETIMEOUT: its outputs are not valid).  All calls of
    the process on the device report to the same check, whatever their stream or
    thread; what one sets while a check runs is left for the next."""
    device = torch.device("cuda" if device is None else device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    torch.cuda.synchronize(device)
    word = _status(device)
    with torch.cuda.device(device):
        taken = torch.empty(1, dtype=torch.int32, device=device)
        A.zero_loss_take_status(word, taken)
        bits = int(taken.item())
    if bits & A.ZERO_LOSS_TIMEOUT:
        raise A.ZeroError(A.ZERO_ETIMEOUT, "check_losses", "a bounded device wait gave up")
    if bits & A.ZERO_LOSS_BAD_TARGET:
        raise A.ZeroError(A.ZERO_EINVAL, "check_losses", "a target lies outside the vocabulary")


# ---- residual addition + RMS norm ---------------------------------------------

def _norm_inputs(where, x, residual, weight):
    rows, dim, xs = _matrix(where, "x", x)
    rs = 0 if residual is None else _matrix(where, "residual", residual, x.dtype, (rows, dim))[2]
    _vector(where, "weight", weight, dim, x.dtype)
    return rows, dim, xs, rs


def residual_norm(x, residual, weight, eps, stream=None):
    """(out, sum): sum = x + residual (residual None: x), out = sum * rstd * weight
    with rstd = (mean(sum^2) + eps)^(-1/2) over each row."""
    rows, dim, xs, rs = _norm_inputs("residual_norm", x, residual, weight)
    with _on(stream):
        out, total = _like(x), _like(x)
        _call("zero_norm_forward", x.data_ptr(), xs, _addr(residual), rs, weight.data_ptr(), eps, rows, dim,
              _LP[x.dtype], out.data_ptr(), dim, total.data_ptr(), dim, A._stream(stream))
    return out, total


def residual_norm_quantized(x, residual, weight, eps, fmt=A.ZERO_QUANT_INT8, stream=None):
    """(codes, scales, sum): residual_norm's out as int8 or E4M3 codes (one byte
    each, int8 tensor) with a float scale per block of 128 elements of a row.
    The scale is NaN, and so all of the block once dequantized, where out has a NaN."""
    rows, dim, xs, rs = _norm_inputs("residual_norm_quantized", x, residual, weight)
    with _on(stream):
        codes = torch.empty((rows, dim), dtype=torch.int8, device=x.device)
        scales = torch.empty((rows, -(-dim // A.ZERO_QUANT_BLOCK)), dtype=torch.float32, device=x.device)
        total = _like(x)
        _call("zero_norm_forward_quantized", x.data_ptr(), xs, _addr(residual), rs, weight.data_ptr(), eps, rows,
              dim, _LP[x.dtype], fmt, codes.data_ptr(), scales.data_ptr(), total.data_ptr(), dim, A._stream(stream))
    return codes, scales, total


def dequantize_rows(codes, scales, fmt, dtype, stream=None):
    """code * scale of its block, in `dtype`, for residual_norm_quantized's outputs."""
    where = "dequantize_rows"
    device = torch._C._cuda_getDevice()
    if codes.ndim != 2 or codes.dtype != torch.int8 or codes.get_device() != device or not codes.is_contiguous():
        _refuse(where, "codes must be a contiguous 2-D int8 tensor on the current CUDA device")
    rows, dim = codes.shape
    if (dtype not in _LP or scales.dtype != torch.float32 or scales.get_device() != device
            or scales.shape != (rows, -(-dim // A.ZERO_QUANT_BLOCK)) or not scales.is_contiguous()):
        _refuse(where, "scales must be one float32 per block of a row, dtype float16 or bfloat16")
    with _on(stream):
        out = torch.empty((rows, dim), dtype=dtype, device=codes.device)
        _call("zero_dequantize_rows", codes.data_ptr(), scales.data_ptr(), fmt, rows, dim, _LP[dtype],
              out.data_ptr(), dim, A._stream(stream))
    return out


def residual_norm_backward(total, weight, grad_out, grad_sum, eps, stream=None):
    """(grad_in, grad_weight) of residual_norm: total is its second output, grad_out
    the gradient of its first, grad_sum (or None) what reaches the sum by its
    other uses.  grad_in is the gradient of x and of residual alike."""
    where = "residual_norm_backward"
    rows, dim, ts = _matrix(where, "total", total)
    _vector(where, "weight", weight, dim, total.dtype)
    gs = _matrix(where, "grad_out", grad_out, total.dtype, (rows, dim))[2]
    ss = 0 if grad_sum is None else _matrix(where, "grad_sum", grad_sum, total.dtype, (rows, dim))[2]
    with _on(stream):
        grad_in, grad_weight = _like(total), _like(weight)
        need = A.zero_norm_backward_workspace(rows, dim)
        space = _scratch(need, total.device)
        _call("zero_norm_backward", total.data_ptr(), ts, weight.data_ptr(), grad_out.data_ptr(), gs, _addr(grad_sum),
              ss, eps, rows, dim, _LP[total.dtype], grad_in.data_ptr(), dim, grad_weight.data_ptr(),
              space.data_ptr(), need, A._stream(stream))
    return grad_in, grad_weight


# ---- cross entropy against the vocabulary matrix --------------------------------

def _loss_inputs(where, hidden, weight, targets):
    tokens, dim, hs = _matrix(where, "hidden", hidden)
    vocab, wide, ws = _matrix(where, "weight", weight, hidden.dtype)
    if wide != dim:
        _refuse(where, "weight has rows of %d, hidden of %d" % (wide, dim))
    _vector(where, "targets", targets, tokens, torch.int64)
    return tokens, dim, vocab, hs, ws


def linear_loss(hidden, weight, targets, ignore=-100, stream=None):
    """(loss, lse), float32 per token: the softmax cross entropy of hidden @ weight.T
    (weight: [vocab, dim]) against int64 targets, and the log-sum-exp the
    backward call takes.  The logits are never stored.  0 where a target is
    `ignore`; see check_losses for targets outside the vocabulary."""
    tokens, dim, vocab, hs, ws = _loss_inputs("linear_loss", hidden, weight, targets)
    device = hidden.device
    status = _status(device)
    with _on(stream):
        loss = torch.empty(tokens, dtype=torch.float32, device=device)
        lse = torch.empty_like(loss)
        need = A.zero_loss_workspace(tokens, vocab, dim)[0]
        space = _scratch(need, device)
        _call("zero_loss_forward", hidden.data_ptr(), hs, weight.data_ptr(), ws, targets.data_ptr(), ignore, tokens,
              vocab, dim, _LP[hidden.dtype], loss.data_ptr(), lse.data_ptr(), status.data_ptr(), space.data_ptr(),
              need, A._stream(stream))
    return loss, lse


def linear_loss_backward(hidden, weight, targets, lse, grad_loss, ignore=-100, grad_hidden=None,
                         grad_weight=None, stream=None):
    """(grad_hidden, grad_weight) of sum(grad_loss * loss), written into the given
    tensors if there are any.  These need 16-byte aligned rows like every matrix,
    which a view of a flat buffer has where the tensor's offset and row length are
    multiples of 8; other gradients go there by clip_gradients."""
    where = "linear_loss_backward"
    tokens, dim, vocab, hs, ws = _loss_inputs(where, hidden, weight, targets)
    _vector(where, "lse", lse, tokens, torch.float32)
    _vector(where, "grad_loss", grad_loss, tokens, torch.float32)
    status = _status(hidden.device)
    with _on(stream):
        if grad_hidden is None:
            grad_hidden = _like(hidden)
        if grad_weight is None:
            grad_weight = _like(weight)
        ghs = _matrix(where, "grad_hidden", grad_hidden, hidden.dtype, (tokens, dim))[2]
        gws = _matrix(where, "grad_weight", grad_weight, hidden.dtype, (vocab, dim))[2]
        need = A.zero_loss_workspace(tokens, vocab, dim)[1]
        space = _scratch(need, hidden.device)
        _call("zero_loss_backward", hidden.data_ptr(), hs, weight.data_ptr(), ws, targets.data_ptr(), ignore, tokens,
              vocab, dim, _LP[hidden.dtype], lse.data_ptr(), grad_loss.data_ptr(), grad_hidden.data_ptr(), ghs,
              grad_weight.data_ptr(), gws, status.data_ptr(), space.data_ptr(), need, A._stream(stream))
    return grad_hidden, grad_weight


# ---- global norm, clipping, packing ----------------------------------------------

_T = torch.Tensor
_DTYPE = attrgetter("dtype")


def _gather(where, name, tensors, dtype, device):
    """(element counts, addresses) of contiguous tensors of one type on the current device."""
    if (set(map(_DTYPE, tensors)) != {dtype} or set(map(_T.get_device, tensors)) != {device}
            or not all(map(_T.is_contiguous, tensors))):
        _refuse(where, "%s must be contiguous tensors of one type (float16, bfloat16 or float32) on the current "
                       "CUDA device" % name)
    return array("q", map(_T.numel, tensors)), array("Q", map(_T.data_ptr, tensors))


def clip_gradients(grads, out=None, offsets=None, max_norm=0.0, loss_scale=1.0, stream=None):
    """(norm, coef, nonfinite), one-element device tensors: the global L2 norm of
    the contiguous gradient tensors `grads` (divided by loss_scale), the clipping
    coefficient, and whether an element is not finite.  The gradients times coef
    go to `out`: None writes them in place; a list takes one tensor each; a 1-D
    tensor is a flat buffer that takes them at `offsets` (elements; default: back
    to back, as ZeroPlan.tensor_offsets lays them out).  Gradients that a step
    averages over ranks are packed with max_norm 0, as they are: the step clips
    the average."""
    where = "clip_gradients"
    if not grads:
        _refuse(where, "no gradients")
    dtype, device = grads[0].dtype, torch._C._cuda_getDevice()
    if dtype not in _CLIP:
        _refuse(where, "grads must be float16, bfloat16 or float32")
    lens, src = _gather(where, "grads", grads, dtype, device)
    n = len(lens)
    if out is None:
        dst = src
    elif isinstance(out, torch.Tensor):
        if out.ndim != 1 or out.dtype != dtype or out.get_device() != device or not out.is_contiguous():
            _refuse(where, "out must be a contiguous 1-D tensor of the gradients' type and device")
        size, first, room = out.element_size(), out.data_ptr(), out.numel()
        if offsets is None and n <= 64:   # a short list costs less than numpy's calls
            at = list(accumulate(lens, initial=0))
            fits = at[n] <= room
            dst = array("Q", [first + size * o for o in at])
        else:
            sizes = np.frombuffer(lens, np.int64)
            at = np.cumsum(sizes) - sizes if offsets is None else np.asarray(offsets, np.int64)
            fits = at.shape == (n,) and at.min() >= 0 and (at + sizes).max() <= room
            dst = array("Q", (at * size + first).tobytes()) if fits else None
        if not fits:
            _refuse(where, "a gradient does not fit into out at its offset")
    else:
        into, dst = _gather(where, "out", out, dtype, device)
        if into != lens:
            _refuse(where, "out must hold one tensor of the same length per gradient")
    with _on(stream):
        at_lens, need = lens.buffer_info()[0], _i64()
        _call("zero_clip_workspace", n, at_lens, byref(need))
        found = torch.empty(3, dtype=torch.float32, device=grads[0].device)
        norm, coef, nonfinite = found.unbind()
        nonfinite = nonfinite.view(torch.int32)
        space = _scratch(need.value, grads[0].device)
        at = found.data_ptr()
        _call("zero_clip_gradients", n, src.buffer_info()[0], at_lens, _CLIP[dtype], dst.buffer_info()[0], loss_scale,
              max_norm, at, at + 4, at + 8, space.data_ptr(), need.value, A._stream(stream))
    return norm, coef, nonfinite
