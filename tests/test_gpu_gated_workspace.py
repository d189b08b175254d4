"""The gated projections' backward call with a workspace on any 16-byte boundary, which is all that the header asks for:
the same bits as from one on a boundary of 1024, whatever the workspace held, and nothing written outside it."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# few tokens and whole tiles, each with grad_x in one sum and in several; widths on a sector and off it
@pytest.mark.parametrize("t,d,f", [(3, 72, 136), (3, 72, 1000), (40, 264, 1000), (129, 72, 136), (300, 72, 1000), (300, 264, 520)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_any_16_bytes(t, d, f, dtype):
    gen = torch.Generator(device="cuda").manual_seed(t + d + f)
    x, gate, up, grad = ((torch.randn(n, m, generator=gen, device="cuda") * s).to(dtype)
                         for n, m, s in ((t, d, 1.0), (f, d, 0.1), (f, d, 0.1), (t, f, 1e-2)))
    want = Z.gated_linear_backward(x, gate, up, grad)
    need = Z.zero_gated_workspace(t, f, d)[1]
    status = torch.zeros(1, device="cuda", dtype=torch.int32)
    guard = 1024
    for off in (0, 16, 32, 48, 112):
        space = torch.full((need + 2 * guard + 1024,), 0xFF, device="cuda", dtype=torch.uint8)   # NaN in every type
        start = guard + (-space.data_ptr() - guard) % 1024 + off
        got = [torch.empty_like(w) for w in want]
        Z.zero_gated_backward(x, d, gate, d, up, d, Z.ZERO_ACT_SILU, grad, f, t, f, d, Z.ZERO_BF16 if dtype == BF else Z.ZERO_FP16,
                              got[0], d, got[1], d, got[2], d, status, space.data_ptr() + start, need)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), off
        assert (space[:start] == 0xFF).all() and (space[start + need:] == 0xFF).all()
    assert int(status) == 0
