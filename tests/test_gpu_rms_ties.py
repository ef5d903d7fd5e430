"""hq_rms_norm's codes on ties that no power of two makes: half of a row's largest value is
63.5 of its scale whatever that value is, and goes to the even code 64, though largest / 127
is no float and largest / 2 over it may come out on either side of 63.5 in 64 bits. The
reference is in whole numbers. Every bf16 mantissa, sums of two values, with and without
gamma, and values one unit beside the tie."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT

pytestmark = pytest.mark.gpu


def whole_codes(n):
    """round(127 n / max |n|), half to even, for whole numbers n of up to 2^40 in each row."""
    top = n.abs().amax(1, keepdim=True).clamp_min(1)
    a = n.abs()
    q = (254 * a) // (2 * top)
    twice = 254 * a - (2 * q + 1) * top    # over or under q + 1/2
    return (torch.sign(n) * (q + ((twice > 0) | ((twice == 0) & (q % 2 == 1))).long())).to(torch.int8)


def check(n, dt, scale, gamma=None, r=None):
    x = (n.double() * scale).to(DT[dt])
    assert torch.equal(x.double(), n.double() * scale)
    h, res = n, None
    if r is not None:
        res = (r.double() * scale).to(DT[dt])
        assert torch.equal(res.double(), r.double() * scale)
        h = n + r
    g = None if gamma is None else gamma.float()
    o = hq.rms_norm(hq.RmsNormDesc(n.shape[1], 1e-6, hq.HQ_RMS_CODES, dt), x, g, res)
    want = whole_codes(h if gamma is None else h * gamma[None, :])
    assert torch.equal(o.codes, want), f"{int((o.codes != want).sum())} codes differ"


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C", [8, 72, 264, 512, 1024, 1152, 2048, 4096, 8192])
def test_half_of_the_largest(C, dt):
    top = torch.arange(128, 256, device="cuda").repeat_interleave(2)    # every bf16 mantissa, two rows each
    g = torch.Generator(device="cuda")
    g.manual_seed(C)
    n = torch.randint(-127, 128, (256, C), generator=g, device="cuda")
    n = torch.where(n.abs() * 2 > top[:, None], torch.zeros_like(n), n)
    n[:, C // 2], n[:, 1], n[:, C - 1] = top * 2, top, -top
    for scale in (1.0, 2.0 ** -9, 2.0 ** 100, 2.0 ** -120):
        check(n, dt, scale)
        check(n * (1 - 2 * (torch.arange(256, device="cuda") % 2))[:, None], dt, scale)
        check(n, dt, scale, gamma=torch.full((C,), 4, device="cuda"))
    if dt == hq.F32:   # one unit beside the tie, of a largest value of 2^20 to 2^21
        m = n * 4096
        m[:, 1] += 1
        m[:, C - 1] += 1
        check(m, dt, 1.0)
        check(m, dt, 2.0 ** -140)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C", [72, 1152, 4096])
def test_ties_of_sums_and_products(C, dt):
    # h = x + r with 12 bits, gamma with 5: the largest and the ties are products of both
    g = torch.Generator(device="cuda")
    g.manual_seed(C + 1)
    for _ in range(4):
        x, r = torch.randint(-15, 16, (300, C), generator=g, device="cuda") * 128, torch.randint(-60, 61, (300, C), generator=g, device="cuda")
        gamma = 2 * torch.randint(1, 16, (C,), generator=g, device="cuda")
        gamma[:2] = torch.tensor([32, 16])
        x[:, 0], r[:, 0] = 15 * 128, torch.randint(61, 128, (300,), generator=g, device="cuda")   # the largest h times the largest gamma
        x[:, 1], r[:, 1] = x[:, 0], r[:, 0]                                                       # half of it
        check(x, dt, 2.0 ** -7, gamma, r)
        check(x, dt, 2.0 ** -7, None, r)
