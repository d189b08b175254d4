"""One AdamW step over a list of torch tensors (the zero_adamw_* calls of include/zero.h),
its moments held in 32 or in 8 bits.

    state = adamw_state(params, bits=8)
    adamw_step(params, grads, state, lr, weight_decay=0.01, copies=weights)

params: contiguous float32 CUDA tensors of any shape, updated in place (parameters that
require grad as well: an update is no part of a graph, but counts as one to a backward pass
that saved what it writes); grads: one contiguous tensor each of
the same length, all float16, bfloat16 or float32; copies: one each, all float16 or bfloat16,
that take the rounded parameters.  Any of them may be parts of flat buffers, at any
element.  A state is a tuple of tensors that belong to the caller, so it is saved, moved and
loaded like any other; steps of one state follow each other on a stream.  The calls can be
captured into a graph, whose replays are the following steps.  Wrong types, lengths or
devices raise ZeroError (ZERO_EINVAL) before any device work.
"""
from typing import NamedTuple, Optional

import torch

from . import _abi as A
from .head import _CLIP, _call, _on, _refuse

_T = torch.Tensor
_BLOCK = A.ZERO_QUANT_BLOCK


class AdamWState(NamedTuple):
    """The moments of a list of tensors, each from a multiple of 128 elements on (adamw_offsets).
    bits=32: m and v are float32, without scales.  bits=8: m int8 (E4M3 codes), v uint8 (codes of
    its root), and a float32 scale for every 128 elements of either.  record: two int64, the
    steps taken and a word of the kernel's."""
    m: torch.Tensor
    v: torch.Tensor
    m_scales: Optional[torch.Tensor]
    v_scales: Optional[torch.Tensor]
    record: torch.Tensor


def adamw_offsets(params):
    """Where each tensor's elements begin in a state's m and v, and their length (a list)."""
    return A.zero_adamw_layout([p.numel() for p in params]).tolist()


def adamw_state(params, bits=32, stream=None):
    """A new state, before the first step, on the current device."""
    if bits not in (8, 32):
        _refuse("adamw_state", "bits is %r, expected 8 or 32" % (bits,))
    total = adamw_offsets(params)[-1]
    device = torch.device("cuda", torch.cuda.current_device())
    with _on(stream):
        zeros = lambda n, dtype: torch.zeros(n, dtype=dtype, device=device)  # noqa: E731
        record = zeros(2, torch.int64)
        if bits == 32:
            return AdamWState(zeros(total, torch.float32), zeros(total, torch.float32), None, None, record)
        return AdamWState(zeros(total, torch.int8), zeros(total, torch.uint8), zeros(total // _BLOCK, torch.float32),
                          zeros(total // _BLOCK, torch.float32), record)


def _vector_at(where, name, t, dtype, n, device):
    """The address of one of the state's tensors."""
    if (not isinstance(t, _T) or t.dtype != dtype or t.ndim != 1 or t.numel() != n or t.get_device() != device
            or not t.is_contiguous()):
        _refuse(where, "the state's %s must be %d contiguous %s on the current CUDA device" % (name, n, dtype))
    return t.data_ptr()


def adamw_step(params, grads, state, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, copies=None, loss_scale=1.0,
               coef=None, skip=None, seed=0, stream=None):
    """One step of every tensor, in place:
      g' = grad * coef / loss_scale,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
      p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps),  copy = p rounded
    t counts the state's steps, on the device.  coef (one float32) and skip (one int32: not 0 leaves
    everything as it was, the count too) are device tensors such as gradient_norm gives; None: 1 and
    never.  seed: of the random rounding of 8-bit moments, which also depends on t and the element."""
    A.tensors().adamw_step(params, grads, copies, state, lr, beta1, beta2, eps, weight_decay, loss_scale, coef, skip, seed,
                           torch._C._cuda_getDevice(), A._stream(stream))


def adamw_moments(state, dtype=torch.float32, stream=None):
    """(m, v) of an 8-bit state as numbers of `dtype`, laid out like the state (adamw_offsets); of a
    32-bit state the state's own tensors, or rounded ones."""
    where = "adamw_moments"
    if dtype not in _CLIP:
        _refuse(where, "dtype must be float16, bfloat16 or float32")
    m, v, m_scales, v_scales, _ = state
    total, device = m.numel(), torch._C._cuda_getDevice()
    if total % _BLOCK:
        _refuse(where, "a state's length is a multiple of %d" % _BLOCK)
    eight = m.dtype == torch.int8
    at = [_vector_at(where, "m", m, torch.int8 if eight else torch.float32, total, device),
          _vector_at(where, "v", v, torch.uint8 if eight else torch.float32, total, device)]
    with _on(stream):
        if not eight:
            return m.to(dtype), v.to(dtype)
        at += [_vector_at(where, n, t, torch.float32, total // _BLOCK, device) for n, t in (("m_scales", m_scales), ("v_scales", v_scales))]
        m_out, v_out = (torch.empty(m.shape, dtype=dtype, device=m.device) for _ in range(2))
        _call("zero_adamw_values", *at, total, _CLIP[dtype], m_out.data_ptr(), v_out.data_ptr(), A._stream(stream))
    return m_out, v_out
