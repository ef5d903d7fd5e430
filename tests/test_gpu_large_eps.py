"""hq_rms_norm and the head norm of hq_rope with an eps so large that it and the mean of
squares, both finite, sum past the largest float: the result is x gamma / sqrt(mean +
eps), not 0. Tolerance: that of ordinary rows (test_gpu_rms_small.py), and the reciprocal
root of a rescaled sum has four roundings (the scaled eps, the sum, the root, the
quotient) in place of one of two units."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import U32, assert_within

pytestmark = pytest.mark.gpu

EPS = 3.4e38


@pytest.mark.parametrize("C", [40, 264, 512, 1152, 4096])
def test_rms_norm(C):
    g = torch.Generator(device="cuda")
    g.manual_seed(C)
    x = torch.randn(12, C, generator=g, device="cuda")
    x[0] = 0.0
    x[0, C // 2] = 1.5e19             # its square is finite, with eps it is not
    x[1] *= 1e19 / C ** 0.5           # a mean below eps, a finite sum
    x[2] *= 1e19                      # a sum of squares past the largest float already
    x[3] *= 1e30
    gamma = 1.0 + 0.2 * torch.randn(C, generator=g, device="cuda")
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    for outputs in (hq.HQ_RMS_Y, hq.HQ_RMS_Y | hq.HQ_RMS_CODES):
        o = hq.rms_norm(hq.RmsNormDesc(C, EPS, outputs), x, gamma)
        h = x.double()
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * gamma.double()
        assert_within(o.y, y, 32 * U32 * y.abs() + 2.0 ** -126, f"C={C}")
        assert o.y[0].any() and o.y[1].any()
        if o.codes is not None:
            s = y.abs().amax(1, keepdim=True) / 127.0
            assert_within(o.scales[:, None], s, 34 * U32 * s + 2.0 ** -149, f"C={C} scales")
            v = h * gamma.double()
            assert torch.equal(o.codes, torch.round(v / (v.abs().amax(1, keepdim=True) / 127.0)).to(torch.int8))


@pytest.mark.parametrize("dim,pairs", [(64, (16, 16)), (72, (18, 18)), (128, (64,)), (16, (4,))])
@pytest.mark.parametrize("layout", [hq.HQ_ROPE_PAIRS, hq.HQ_ROPE_HALVES])
def test_rope(layout, dim, pairs):
    g = torch.Generator(device="cuda")
    g.manual_seed(dim)
    T, heads, P = 5, 3, sum(pairs)
    x = torch.randn(T, heads, dim, generator=g, device="cuda")
    x[0] = 0.0
    x[0, :, dim // 2] = 1.5e19
    x[1] *= 1e19 / dim ** 0.5
    x[2, 1] *= 1e19                   # a large head beside ordinary ones
    x[3] *= 1e30
    gamma = 1.0 + 0.2 * torch.randn(dim, generator=g, device="cuda")
    desc = hq.RopeDesc(heads, 0, dim, pairs, layout, norm=True, eps=EPS)
    pos = torch.zeros(T, len(pairs), dtype=torch.int32, device="cuda")   # no turn: the norm alone
    Y = hq.rope(desc, x.view(T, -1), pos, hq.rope_freqs(desc), gamma).view(T, heads, dim)
    h = x.double()
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    y = h / torch.sqrt(h.square().mean(2, keepdim=True) + eps) * gamma.double()
    assert_within(Y.view(T, -1), y.view(T, -1), 32 * U32 * y.abs().view(T, -1) + 2.0 ** -120)
    assert Y[0].any() and Y[1].any()
