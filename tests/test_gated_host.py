"""The gated projections' calls on the host (CPU only: no kernel is launched): every argument that a call refuses, with
its status, before any CUDA call; the workspace sizes."""
import pytest

import zero_partitioned_mixed_flat_gb300 as Z

P = 1 << 20          # an aligned address that is never read
INVALID, ALIGN = Z.ZERO_EINVAL, Z.ZERO_EALIGN


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_partitioned_mixed_flat_gb300 import build
    build.build()
    return Z.load()


def refused(code, call, args, changed):
    assert not set(changed) - set(args)
    with pytest.raises(Z.ZeroError) as e:
        call(*{**args, **changed}.values(), stream=0)
    assert e.value.code == code, (changed, str(e.value))
    assert Z.zero_last_error()


FORWARD = dict(x=P, x_stride=64, gate=P, gate_stride=64, up=P, up_stride=64, act=0, n_tokens=40, wide=72, dim=64, lp=1,
               out=P, out_stride=72, status=P, workspace=P, workspace_bytes=1 << 40)
BACKWARD = dict(x=P, x_stride=64, gate=P, gate_stride=64, up=P, up_stride=64, act=0, grad_out=P, grad_out_stride=72,
                n_tokens=40, wide=72, dim=64, lp=1, grad_x=P, grad_x_stride=64, grad_gate=P, grad_gate_stride=64, grad_up=P,
                grad_up_stride=64, status=P, workspace=P, workspace_bytes=1 << 40)
BOTH = [(INVALID, dict(n_tokens=-1)), (INVALID, dict(n_tokens=2 ** 31 - 2 ** 16)), (INVALID, dict(dim=0)),
        (INVALID, dict(dim=Z.ZERO_HEAD_MAX_DIM + 8)), (ALIGN, dict(dim=60)), (INVALID, dict(lp=2)), (INVALID, dict(act=3)),
        (INVALID, dict(act=-1)), (INVALID, dict(wide=0)), (INVALID, dict(wide=1 << 30)), (ALIGN, dict(wide=68)),
        (INVALID, dict(status=None)), (ALIGN, dict(status=P + 2)), (ALIGN, dict(workspace=P + 8))]


def strides(names):
    return [(code, {n + "_stride": v}) for n in names for code, v in ((INVALID, 56), (ALIGN, 76), (INVALID, (1 << 40) + 8))]


def pointers(names):
    return [c for n in names for c in ((INVALID, {n: None}), (ALIGN, {n: P + 8}))]


@pytest.mark.parametrize("code,changed", BOTH + strides(["x", "gate", "up", "out"]) + pointers(["x", "gate", "up", "out"]))
def test_forward_refuses(code, changed):
    refused(code, Z.zero_gated_forward, FORWARD, changed)


MATRICES = ["x", "gate", "up", "grad_out", "grad_x", "grad_gate", "grad_up"]


@pytest.mark.parametrize("code,changed", BOTH + strides(MATRICES) + pointers(MATRICES) + [
    (INVALID, dict(workspace=None)), (INVALID, dict(workspace_bytes=1024))])
def test_backward_refuses(code, changed):
    refused(code, Z.zero_gated_backward, BACKWARD, changed)


def test_a_forward_call_refuses_a_short_workspace():
    need = Z.zero_gated_workspace(40, 72, 64)[0]
    if need:
        refused(INVALID, Z.zero_gated_forward, FORWARD, dict(workspace_bytes=need - 1))


def test_no_token_needs_no_rows():
    Z.zero_gated_forward(*{**FORWARD, "n_tokens": 0, "x": None, "out": None}.values(), stream=0)


def test_workspace_sizes():
    for t in (0, 1, 5, 64, 300, 5000):
        for wide, dim in ((8, 8), (136, 72), (11000, 4096)):
            forward, backward = Z.zero_gated_workspace(t, wide, dim)
            assert forward >= 0 and backward >= 2 * t * wide * 2
    # both slopes, and at most 16 float sums of the tiles' rows
    assert Z.zero_gated_workspace(4096, 10928, 4096)[1] <= 2 * 4096 * 10928 * 2 + 4 * 4096 * 4096 * 4 + 8192


def test_the_tensor_call_refuses_what_is_no_cuda_matrix():
    """Before any CUDA call: the module that takes torch tensors."""
    import torch
    call = Z._abi.tensors().gated_forward
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    for bad in (x, x.float(), x[0], None, 3, x.to_sparse()):
        with pytest.raises(Z.ZeroError) as e:
            call(bad, x, x, 0, 0, P, 0)
        assert e.value.code == INVALID
    with pytest.raises(Z.ZeroError, match="requires grad"):
        call(torch.zeros(2, 8, requires_grad=True), x, x, 0, 0, P, 0)
    with pytest.raises(TypeError):
        call(x, x)
