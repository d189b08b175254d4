"""The training-head calls of include/zero.h on the host (CPU only: no kernel is
launched): every argument that a call refuses, with its status and a message,
before any CUDA call; the workspace sizes."""
import numpy as np
import pytest

import zero_partitioned_mixed_flat_gb300 as Z
from zero_partitioned_mixed_flat_gb300 import _abi as A

P = 1 << 20          # an aligned address that is never read
Q = P + 4096
INVALID, ALIGN = Z.ZERO_EINVAL, Z.ZERO_EALIGN


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_partitioned_mixed_flat_gb300 import build
    build.build()
    return Z.load()


def refused(code, call, args, changed):
    a = dict(args)
    unknown = set(changed) - set(a)
    assert not unknown
    a.update(changed)
    with pytest.raises(Z.ZeroError) as e:
        call(*a.values(), stream=0)
    assert e.value.code == code, (changed, str(e.value))
    assert Z.zero_last_error()


NORM = dict(x=P, x_stride=64, residual=Q, residual_stride=64, weight=P, eps=1e-5, n_rows=4, dim=64, lp=1,
            out=P, out_stride=64, sum_out=Q, sum_stride=64)
MATRIX = [(INVALID, {"%s_stride": 56}), (ALIGN, {"%s_stride": 68})]


def strides_of(names):
    return [(code, {k % n: v for k, v in d.items()}) for n in names for code, d in MATRIX]


SHAPE = [(INVALID, dict(n_rows=-1)), (INVALID, dict(n_rows=2 ** 31 - 2 ** 16)), (INVALID, dict(dim=0)),
         (INVALID, dict(dim=Z.ZERO_HEAD_MAX_DIM + 8)), (ALIGN, dict(dim=60)), (INVALID, dict(lp=2))]


@pytest.mark.parametrize("code,changed", SHAPE + strides_of(["x", "residual", "out", "sum"]) + [
    (INVALID, dict(x=None)), (INVALID, dict(weight=None)), (INVALID, dict(out=None)), (ALIGN, dict(x=P + 8)),
    (ALIGN, dict(residual=P + 2)), (ALIGN, dict(weight=P + 8)), (ALIGN, dict(out=P + 4)), (ALIGN, dict(sum_out=P + 8)),
    (INVALID, dict(eps=-1e-6)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))),
])
def test_norm_forward_refuses(code, changed):
    refused(code, Z.zero_norm_forward, NORM, changed)


QUANT = dict(x=P, x_stride=64, residual=None, residual_stride=0, weight=P, eps=1e-5, n_rows=4, dim=64, lp=0, fmt=1,
             codes=P, scales=Q, sum_out=None, sum_stride=0)


@pytest.mark.parametrize("code,changed", SHAPE + strides_of(["x"]) + [
    (INVALID, dict(fmt=2)), (INVALID, dict(codes=None)), (INVALID, dict(scales=None)), (ALIGN, dict(codes=P + 8)),
    (ALIGN, dict(scales=P + 4)), (INVALID, dict(eps=-1.0)),
])
def test_norm_forward_quantized_refuses(code, changed):
    refused(code, Z.zero_norm_forward_quantized, QUANT, changed)


DEQUANT = dict(codes=P, scales=Q, fmt=0, n_rows=4, dim=64, lp=1, out=P, out_stride=64)


@pytest.mark.parametrize("code,changed", SHAPE + strides_of(["out"]) + [
    (INVALID, dict(fmt=-1)), (INVALID, dict(codes=None)), (ALIGN, dict(scales=P + 4)), (INVALID, dict(out=None)),
])
def test_dequantize_refuses(code, changed):
    refused(code, Z.zero_dequantize_rows, DEQUANT, changed)


BACK = dict(sum_in=P, sum_stride=64, weight=P, grad_out=Q, grad_out_stride=64, grad_sum=P, grad_sum_stride=64, eps=1e-5,
            n_rows=4, dim=64, lp=1, grad_in=Q, grad_in_stride=64, grad_weight=P, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("code,changed", SHAPE + strides_of(["sum", "grad_out", "grad_sum", "grad_in"]) + [
    (INVALID, dict(sum_in=None)), (INVALID, dict(grad_out=None)), (INVALID, dict(grad_in=None)),
    (INVALID, dict(grad_weight=None)), (ALIGN, dict(grad_weight=P + 2)), (INVALID, dict(workspace=None)),
    (ALIGN, dict(workspace=P + 8)), (INVALID, dict(workspace_bytes=0)), (INVALID, dict(eps=float("nan"))),
])
def test_norm_backward_refuses(code, changed):
    refused(code, Z.zero_norm_backward, BACK, changed)


LOSS = dict(hidden=P, hidden_stride=64, weight=Q, weight_stride=64, target=P, ignore=-100, n_tokens=4, vocab=10, dim=64,
            lp=0, loss=P, lse=Q, status=P, workspace=P, workspace_bytes=1 << 30)
LOSS_SHAPE = [(c, {k.replace("n_rows", "n_tokens"): v for k, v in d.items()}) for c, d in SHAPE] + [
    (INVALID, dict(vocab=0)), (INVALID, dict(vocab=2 ** 31 - 2 ** 16)), (INVALID, dict(hidden=None)),
    (INVALID, dict(weight=None)), (INVALID, dict(target=None)), (ALIGN, dict(target=P + 4)), (INVALID, dict(status=None)),
    (ALIGN, dict(status=P + 2)), (INVALID, dict(workspace=None)), (ALIGN, dict(workspace=P + 8)),
    (INVALID, dict(workspace_bytes=16)), (ALIGN, dict(hidden=P + 8)), (ALIGN, dict(weight=P + 8))] + strides_of(["hidden", "weight"])


@pytest.mark.parametrize("code,changed", LOSS_SHAPE + [(INVALID, dict(loss=None)), (INVALID, dict(lse=None)),
                                                       (ALIGN, dict(loss=P + 4))])
def test_loss_forward_refuses(code, changed):
    refused(code, Z.zero_loss_forward, LOSS, changed)


LOSS_BACK = dict(hidden=P, hidden_stride=64, weight=Q, weight_stride=64, target=P, ignore=-100, n_tokens=4, vocab=10,
                 dim=64, lp=0, lse=P, grad_loss=Q, grad_hidden=P, grad_hidden_stride=64, grad_weight=Q,
                 grad_weight_stride=64, status=P, workspace=P, workspace_bytes=1 << 30)


@pytest.mark.parametrize("code,changed", LOSS_SHAPE + strides_of(["grad_hidden", "grad_weight"]) + [
    (INVALID, dict(lse=None)), (INVALID, dict(grad_loss=None)), (INVALID, dict(grad_hidden=None)),
    (INVALID, dict(grad_weight=None)), (ALIGN, dict(grad_weight=P + 8)), (ALIGN, dict(grad_loss=P + 4)),
])
def test_loss_backward_refuses(code, changed):
    refused(code, Z.zero_loss_backward, LOSS_BACK, changed)


CLIP = dict(grads=[P, Q], lens=[5, 7], dtype=2, out=[P, Q], loss_scale=1.0, max_norm=1.0, norm=P, coef=P, nonfinite=P,
            workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("code,changed", [
    (INVALID, dict(lens=[5, -1])), (INVALID, dict(lens=[5, 2 ** 41])), (INVALID, dict(dtype=3)),
    (INVALID, dict(loss_scale=0.0)), (INVALID, dict(loss_scale=float("inf"))), (INVALID, dict(max_norm=float("nan"))),
    (INVALID, dict(grads=[P, None])), (INVALID, dict(out=[None, Q])), (ALIGN, dict(grads=[P + 2, Q])),
    (ALIGN, dict(out=[P, Q + 1])), (ALIGN, dict(dtype=0, grads=[P + 1, Q])), (ALIGN, dict(norm=P + 2)),
    (ALIGN, dict(nonfinite=P + 1)), (INVALID, dict(workspace=None)), (INVALID, dict(workspace_bytes=8)),
    (ALIGN, dict(workspace=P + 8)),
])
def test_clip_refuses(code, changed):
    refused(code, Z.zero_clip_gradients, CLIP, changed)


def test_clip_lists_of_other_lengths():
    with pytest.raises(ValueError):
        Z.zero_clip_gradients([P], [1, 2], 2, None, 1.0, 1.0, P, P, P, P, 1 << 20, stream=0)


def test_wait_limit_refuses():
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_loss_set_wait_limit(-1)
    assert e.value.code == INVALID


def test_workspaces():
    """Sizes grow with the shape, are whole and small next to the logits."""
    assert Z.zero_norm_backward_workspace(0, 64) == 0
    for rows, dim in ((1, 8), (1023, 768), (100000, 4096), (5, 16384)):
        need = Z.zero_norm_backward_workspace(rows, dim)
        assert 0 < need <= 64 << 20 and need % 4 == 0
    for tokens, vocab, dim in ((1, 1, 8), (4, 50257, 768), (1023, 50257, 768), (4096, 50257, 4096), (16384, 50257, 4096)):
        fwd, bwd = Z.zero_loss_workspace(tokens, vocab, dim)
        assert fwd > 0 and bwd > 0
        if tokens >= 4096:
            assert fwd < tokens * vocab * 4 / 50        # the statistics of a tile of 256 logits: 8 bytes
            rows = tokens + 256
            # a piece of the slopes, the counted hidden states, and few sums of grad_hidden
            assert bwd < (300 << 20) + rows * dim * (2 + 4 * 4)
    for lens in ([], [0], [1], [10 ** 9] * 4, [3] * 2000):
        need = Z.zero_clip_workspace(np.array(lens, np.int64))
        assert 0 < need < 1 << 20
    with pytest.raises(Z.ZeroError):
        Z.zero_norm_backward_workspace(4, 60)
    with pytest.raises(Z.ZeroError):
        Z.zero_loss_workspace(4, 0, 64)


def test_library_status_names():
    assert (A.ZERO_LOSS_TIMEOUT, A.ZERO_LOSS_BAD_TARGET, A.ZERO_FP32) == (1, 2, 2)


def test_the_package_needs_no_torch_until_the_head_is_used():
    import subprocess
    import sys
    program = ("import sys; sys.modules['torch'] = None\n"
               "import zero_partitioned_mixed_flat_gb300 as Z\n"
               "Z.load(); Z.zero_memory_report(8, 1)\n"
               "try:\n    Z.linear_loss\nexcept ImportError:\n    print('late')\n")
    out = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=120)
    assert out.stdout.strip() == "late", out.stderr
    assert callable(Z.residual_norm) and not hasattr(Z, "no_such_name")
