"""The step over tensors on the host (CPU only: no kernel is launched): the layout, and every argument that a call
refuses, with its status, before any CUDA call."""
import numpy as np
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


STEP = dict(params=[P, P], grads=[P, P], grad_dtype=1, copies=[P, P], copy_type=1, lens=[300, 7], moments=1, m=P, v=P,
            m_scales=P, v_scales=P, record=P, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.1, loss_scale=1.0, coef=P,
            skip=P, seed=0)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("code,changed", [
    (INVALID, dict(params=[P, 0])), (INVALID, dict(grads=[0, P])), (INVALID, dict(copies=[P, 0])),
    (ALIGN, dict(params=[P + 2, P])), (ALIGN, dict(grads=[P, P + 1])), (ALIGN, dict(copies=[P + 1, P])),
    (ALIGN, dict(grads=[P + 2, P], grad_dtype=2)),
    (INVALID, dict(grad_dtype=3)), (INVALID, dict(copy_type=2)), (INVALID, dict(moments=2)), (INVALID, dict(lens=[300, -1])),
    (INVALID, dict(lens=[300, (1 << 40) + 1])), (INVALID, dict(m=None)), (INVALID, dict(v=None)), (INVALID, dict(m_scales=None)),
    (INVALID, dict(v_scales=None)), (ALIGN, dict(m=P + 8)), (ALIGN, dict(v=P + 4)), (ALIGN, dict(m_scales=P + 4)),
    (INVALID, dict(record=None)), (ALIGN, dict(record=P + 4)), (ALIGN, dict(coef=P + 2)), (ALIGN, dict(skip=P + 1)),
    (INVALID, dict(lr=NAN)), (INVALID, dict(lr=INF)), (INVALID, dict(wd=NAN)), (INVALID, dict(eps=-1e-8)), (INVALID, dict(eps=NAN)),
    (INVALID, dict(beta1=1.0)), (INVALID, dict(beta1=-0.1)), (INVALID, dict(beta2=1.5)), (INVALID, dict(beta2=NAN)),
    (INVALID, dict(loss_scale=0.0)), (INVALID, dict(loss_scale=-1.0)), (INVALID, dict(loss_scale=INF)),
])
def test_step_refuses(code, changed):
    refused(code, Z.zero_adamw_step, STEP, changed)


@pytest.mark.parametrize("changed", [dict(lr=1e39), dict(lr=-1e39), dict(eps=1e39), dict(lr=1e30, wd=-1e30),
                                     dict(eps=1e-39), dict(eps=2.0 ** -126 * 0.999)])
def test_step_refuses_numbers_outside_a_float(changed):
    """What is infinite as a float, and an eps whose reciprocal is: a moment of 0 times that is NaN, and not 0."""
    refused(INVALID, Z.zero_adamw_step, STEP, changed)


def test_step_refuses_lists_that_do_not_match():
    with pytest.raises(ValueError):
        Z.zero_adamw_step(*{**STEP, "grads": [P]}.values(), stream=0)


VALUES = dict(m=P, v=P, m_scales=P, v_scales=P, n_elems=256, dtype=2, m_out=P, v_out=P)


@pytest.mark.parametrize("code,changed", [(INVALID, {k: None}) for k in ("m", "v", "m_scales", "v_scales", "m_out", "v_out")]
                         + [(ALIGN, {k: P + 8}) for k in ("m", "v", "m_scales", "v_scales", "m_out", "v_out")]
                         + [(INVALID, dict(dtype=3)), (INVALID, dict(n_elems=-128)), (ALIGN, dict(n_elems=100))])
def test_values_refuses(code, changed):
    refused(code, Z.zero_adamw_values, VALUES, changed)


def test_no_values():
    Z.zero_adamw_values(*{**VALUES, "n_elems": 0, "m": None, "m_out": None}.values(), stream=0)


def test_layout():
    assert Z.zero_adamw_layout([]).tolist() == [0]
    lens = [0, 1, 127, 128, 129, 0, 1 << 40]
    at = Z.zero_adamw_layout(lens)
    assert at.dtype == np.int64 and (at % Z.ZERO_QUANT_BLOCK == 0).all()
    assert (np.diff(at) == [-(-n // 128) * 128 for n in lens]).all()
    with pytest.raises(Z.ZeroError):
        Z.zero_adamw_layout([5, -1])
    with pytest.raises(Z.ZeroError):
        Z.zero_adamw_layout([1 << 40] * 17)


def test_the_tensor_call_refuses_what_is_no_cuda_tensor():
    """Before any CUDA call: the module that takes torch tensors."""
    import torch
    call = Z._abi.tensors().adamw_step
    p = torch.zeros(5)
    numbers = (1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0, None, None)
    for params in ([p], [3], [p.half()], [None], []):
        with pytest.raises(Z.ZeroError) as e:
            call(params, [], None, (None,) * 5, *numbers, 0, 0, 0)
        assert e.value.code == INVALID
    with pytest.raises(TypeError):
        call(p)
    with pytest.raises(TypeError):
        call(5, [p], None, (None,) * 5, *numbers, 0, 0, 0)
    with pytest.raises(Z.ZeroError):
        call([p], [p], None, (None,) * 5, *numbers, 1 << 40, 0, 0)
