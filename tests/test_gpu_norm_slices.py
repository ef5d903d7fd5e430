"""hq_group_norm where one grid does not hold the samples' blocks: the call is cut into
slices, and every sample is what a call of few samples gives."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,P,C,G,dt", [((1 << 20) + 3, 33, 512, 16, hq.BF16), ((1 << 22) + 9, 3, 1024, 1024, hq.BF16)])
def test_many_slabs_of_many_samples(S, P, C, G, dt):
    desc = hq.NormDesc(C, G, 1e-5, hq.HQ_ACT_SILU, dt, dt)
    plan = hq.group_norm_plan(desc, S, P)
    assert plan.kernel == hq.HQ_NORM_BLOCK and plan.slices > 1
    few = torch.randn(1024, P, C, device="cuda").to(torch.bfloat16)
    want = hq.group_norm(desc, few)
    X = torch.empty(S, P, C, dtype=torch.bfloat16, device="cuda")
    whole = S // 1024 * 1024
    X[:whole].view(-1, 1024, P, C).copy_(few.expand(S // 1024, -1, -1, -1))
    X[whole:] = few[:S - whole]
    hq.group_norm(desc, X, out=X)
    for part in X[:whole].view(-1, 1024, P, C):
        assert torch.equal(part, want)
    assert torch.equal(X[whole:], want[:S - whole])
