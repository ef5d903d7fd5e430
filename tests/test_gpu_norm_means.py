"""hq_group_norm's means: a group of equal values is that value's beta bit for bit in
every form, whatever rounds on the way (sums of equal values, a division by a count that
is no power of two), and a mean far from zero costs a few units of itself.

Tolerance of a mean m over values of size up to t (U = 2^-24): the rows in a lane's
registers give their mean to one rounding, corrected by the sum of differences (2 U t);
each join rounds its mean (U t) and its difference times a weight (3 U |d|, d a difference
of two means of the group, no more than 4 std here). At most 16 joins in a block (15
batches of 4 rows and a tree of 2 lanes, or one batch and a tree of 1024), one of the
units and one of the chunks: 20 U t + 240 U std. Then (x - m) / std, gamma, beta and phi
as in test_gpu_norm."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT, U32, assert_within

pytestmark = pytest.mark.gpu

# samples, positions: one launch (256 and 1024 threads, 2 and 8 rows per lane), chunks, chunks joined between
FORMS = [(3, 2), (2, 77), (1, 200), (70, 600), (1, 3000), (1, 6001), (3, 40_001)]
WIDTHS = [(8, 1), (40, 4), (72, 3), (64, 8), (320, 32), (1032, 43), (4096, 4)]


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C,G", WIDTHS)
@pytest.mark.parametrize("S,P", FORMS)
def test_constant_groups_give_beta(S, P, C, G, dt):
    desc = hq.NormDesc(C, G, 1e-12, x_dtype=dt, y_dtype=dt)
    beta = torch.linspace(-1, 1, C, device="cuda")
    for value in (0.1, 1000.1, -1000.25, 3.5, 1.0 / 3.0, -7e-4):
        # each group its own constant
        per = (value * (1.0 + torch.arange(G, device="cuda") / 7.0)).repeat_interleave(C // G)
        X = per.to(DT[dt]).expand(S, P, C).contiguous()
        Y = hq.group_norm(desc, X, None, beta)
        assert torch.equal(Y, beta.to(DT[dt]).expand(S, P, C)), f"{value}: {(Y.float() - beta).abs().max().item()}"


@pytest.mark.parametrize("C,G", WIDTHS)
@pytest.mark.parametrize("S,P", FORMS)
def test_means_far_from_zero(S, P, C, G):
    g = torch.Generator(device="cuda")
    g.manual_seed(S + P + C)
    X = 1000.1 + torch.randn(S, P, C, generator=g, device="cuda")
    x = X.double().view(S, P, G, C // G)
    m = x.mean((1, 3), keepdim=True)
    var = (x - m).square().mean((1, 3), keepdim=True)
    top, std = x.abs().amax((1, 3), keepdim=True), var.sqrt()
    em = 20 * U32 * top + 240 * U32 * std
    rs = 1.0 / torch.sqrt(var + 1e-5)
    z = (x - m) * rs
    # the squares: relative 40 U in their sum, the square of the mean's error
    tol = em * rs + z.abs() * (20 * U32 + 0.5 * (em * rs) ** 2 + 6 * U32)
    Y = hq.group_norm(hq.NormDesc(C, G), X)
    assert_within(Y.view(-1, C), z.reshape(-1, C), tol.expand_as(x).reshape(-1, C) + U32 * z.abs().reshape(-1, C) + 1e-30,
                  f"S={S} P={P} C={C} G={G}")


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C,G", [(64, 8), (512, 1), (1152, 1), (320, 32), (4096, 2)])
@pytest.mark.parametrize("P", [1, 2, 300, 6001])
def test_squares_past_the_largest_float(P, C, G, dt):
    # a group whose variance is no float has an infinite one: phi(beta), not a value the
    # size of the input; the other groups and samples keep theirs
    g = torch.Generator(device="cuda")
    g.manual_seed(P + C)
    X = torch.randn(3, P, C, generator=g, device="cuda").to(DT[dt])
    beta = torch.linspace(-1, 1, C, device="cuda")
    desc = hq.NormDesc(C, G, x_dtype=dt, y_dtype=dt)
    want = hq.group_norm(desc, X, None, beta)
    w = C // G
    X[1, :, :w] = (torch.randn(P, w, generator=g, device="cuda") * 1e30).to(DT[dt])
    want[1, :, :w] = beta[:w].to(DT[dt])
    assert torch.equal(hq.group_norm(desc, X, None, beta), want)
