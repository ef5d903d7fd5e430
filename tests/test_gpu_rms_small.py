"""hq_rms_norm where h gamma or its factors leave the range of normal floats, against
float64: rows whose h gamma is subnormal or below the smallest float (codes, scales and
the norm are those of the unrounded products), alone and beside ordinary rows and rows of
zeros.

Tolerance, in units of 2^-24. h is one rounding. The sum of squares: two of h, 32
additions in a lane (4 pieces of 8), 6 across lanes, 2 across waves; the mean two: 44,
halved by the root, and 2 of the reciprocal root: 24 of rstd. A value of the norm: h, the
product with gamma, rstd and the product with it: 27. A scale: the maximum 2, rstd 24, 1 / 127
and two products: 29. One more for second-order terms. A result below 2^-126 is off by up to
half the smallest float, 2^-150, in each of its two last roundings."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT, U32, assert_within

pytestmark = pytest.mark.gpu

CODES = hq.HQ_RMS_CODES


def rms64(x, r, gamma, eps):
    h = x.double() if r is None else x.double() + r.double()
    g = 1.0 if gamma is None else gamma.double()
    rstd = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    v = h * g
    s = v.abs().amax(1, keepdim=True) / 127.0
    codes = torch.where(s > 0, torch.round(v / s), torch.zeros_like(v)).to(torch.int8)
    return h * rstd * g, codes, s * rstd


def check_codes(x, gamma, eps, what, r=None):
    o = hq.rms_norm(hq.RmsNormDesc(x.shape[1], eps, CODES, hq.F32 if x.dtype is torch.float32 else hq.BF16), x, gamma, r)
    _, codes, scales = rms64(x, r, gamma, eps)
    assert_within(o.scales[:, None], scales, 30 * U32 * scales + 2.0 ** -149, what + " scales")
    assert torch.equal(o.codes, codes), f"{what}: {int((o.codes != codes).sum())} codes differ"


def randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


WIDTHS = [40, 72, 264, 512, 1024, 1152, 2048, 4096, 8192]


@pytest.mark.parametrize("C", WIDTHS)
def test_scales_of_subnormal_rows(C):
    # whole multiples of the smallest float, largest of a row 2^-130 to 2^-149 (one that is all the row has)
    top = 2.0 ** torch.arange(19, -1, -1, device="cuda").float()
    x = (randn(C, 20, C).clamp(-3, 3) / 3 * top[:, None]).round()
    x[:, C // 2] = top
    x = (x.double() * 2.0 ** -149).float()
    check_codes(x, None, 2.0 ** -100, f"C={C}")
    check_codes(torch.cat([x, torch.zeros_like(x), randn(C + 1, 20, C)])[torch.randperm(60)].contiguous(), None, 2.0 ** -100,
                f"C={C} among others")


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", [hq.F32, hq.BF16])
def test_scales_and_codes_of_subnormal_products(C, dt):
    # h gamma of 2^-120 to 2^-200: subnormal in fp32, or nothing
    x, gamma = randn(C, 50, C), randn(C + 1, C) * 2.0 ** -85
    gamma[C // 3] = 0.0
    x = (x * 2.0 ** -torch.linspace(20.0, 100.0, 50, device="cuda")[:, None]).to(DT[dt])
    x[7], x[20] = 0.0, randn(C + 2, C).to(DT[dt])   # beside a row of zeros and an ordinary one
    check_codes(x, gamma, 2.0 ** -100, f"C={C} dt={dt}")
    check_codes(x, gamma, 2.0 ** -100, f"C={C} dt={dt} residual", r=(x.float() * 0.375).to(DT[dt]))
    check_codes(x, torch.zeros_like(gamma), 2.0 ** -100, f"C={C} dt={dt} gamma of zeros")


@pytest.mark.parametrize("C", [72, 1152, 4096])
def test_one_value_below_the_smallest_float(C):
    # every product but one is exactly zero, that one rounds to zero in fp32: it is the row's maximum
    x = torch.zeros(6, C, device="cuda")
    x[1, 3], x[4, C - 1] = 2.0 ** -80, -2.0 ** -90
    gamma = torch.full((C,), 2.0 ** -75, device="cuda")
    check_codes(x, gamma, 2.0 ** -100, f"C={C}")


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", [hq.F32, hq.BF16])
@pytest.mark.parametrize("ydt", [hq.F32, hq.BF16])
def test_norm_of_subnormal_products(C, dt, ydt):
    # h gamma is subnormal or nothing in fp32, the norm an ordinary number (rstd up to 2^50); up to an
    # rstd of 2^24 an error of half the smallest float of h gamma is at most 2^-126 of the norm
    x, gamma = randn(C, 50, C), randn(C + 1, C) * 2.0 ** -85
    x = (x * 2.0 ** -torch.linspace(15.0, 100.0, 50, device="cuda")[:, None]).to(DT[dt])
    x[7], x[20] = 0.0, randn(C + 2, C).to(DT[dt])
    r = (x.float() * 0.375).to(DT[dt])
    for outputs in (hq.HQ_RMS_Y, hq.HQ_RMS_Y | hq.HQ_RMS_SUM | CODES):
        for res in (None, r):
            o = hq.rms_norm(hq.RmsNormDesc(C, 2.0 ** -100, outputs, dt, ydt), x, gamma, res)
            y, _, _ = rms64(x, res, gamma, 2.0 ** -100)
            half = torch.finfo(DT[ydt]).eps / 2
            least = 2.0 ** -126 if ydt == hq.F32 else 2.0 ** -126 + 2.0 ** -134   # bf16's own smallest: 2^-133
            assert_within(o.y, y, (28 * U32 * (1 + half) + half) * y.abs() + least, f"C={C} dt={dt} ydt={ydt} {outputs}")
            big = (x.double() + (0 if res is None else res.double())).square().mean(1) < 2.0 ** -50
            assert big.sum() > 20
            assert_within(o.y[big], y[big], (28 * U32 * (1 + half) + half) * y[big].abs() + (2.0 ** -133 if ydt == hq.BF16 else 2.0 ** -148),
                          f"C={C} dt={dt} ydt={ydt} {outputs} where rstd is past 2^24")
