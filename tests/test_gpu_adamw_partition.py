"""The step over tensors on the partitions of a plan: two ranks' flat partitions, reduced by the plan's own call, each a
list of one with a state of its own, its copy a part of the flat parameter buffer."""
import pytest
import torch

import zero_partitioned_mixed_flat_gb300 as Z

from .test_gpu_adamw import Case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bits", [8, 32])
def test_partitions(bits):
    ranks, scale = 2, 64.0
    plan = Z.ZeroPlan(-1, ranks, [5000, 17, 3001], 128, 2, None, Z.ZERO_BF16)
    P = plan.part_len
    gen = torch.Generator(device="cuda").manual_seed(1)
    params = torch.zeros(plan.psi_padded, device="cuda", dtype=BF)
    cases = []
    for r in range(ranks):
        c = Case([P], bits, F32, BF, key=r)
        c.copies = [params[r * P:(r + 1) * P]]
        cases.append(c)
    for step in range(4):
        flats = [(torch.randn(plan.psi_padded, generator=gen, device="cuda") * scale).to(BF) for _ in range(ranks)]
        if step == 2:
            flats[1][P + 5] = float("inf")     # in the second partition: nobody steps
        for r, c in enumerate(cases):
            plan.reduce(r, [f[r * P:(r + 1) * P] for f in flats], c.grads[0], scale)
        _, coef, bad = Z.gradient_norm([c.grads[0] for c in cases], max_norm=1.0)
        assert int(bad) == (step == 2)
        if step == 2:
            kept = [t.clone() for c in cases for t in (*c.params, *c.copies, *(s for s in c.state if s is not None))]
            for c in cases:
                Z.adamw_step(c.params, c.grads, c.state, 1e-3, copies=c.copies, coef=coef, skip=bad)
            assert all(torch.equal(a, b) for a, b in zip(kept, (t for c in cases for t in (*c.params, *c.copies, *(s for s in c.state if s is not None)))))
            continue
        assert float(coef) < 0.1
        for c in cases:
            c.step(coef=coef, skip=bad)       # element by element against 64 bits, or to the bit
        assert torch.equal(params, torch.cat([c.params[0] for c in cases]).to(BF))
    assert all(int(c.state.record[0]) == 3 for c in cases)
    plan.close()
