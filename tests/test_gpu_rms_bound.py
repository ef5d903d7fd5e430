"""hq_rms_norm against float64 within the error that its own number of roundings allows (the
derivation stands in test_gpu_rms_small.py: 27 units of 2^-24 of the norm and 29 of a scale,
one more for second-order terms), every form and its borders, both types."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT, U32, assert_within
from test_gpu_rms import ALL, WIDTHS, make, rms64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C", WIDTHS)
def test_norm_and_scales(C, dt):
    for T in (1, 7, 300):
        for residual in (True, False):
            x, r, gamma = make(T, C, dt)
            r = r if residual else None
            for outputs in (ALL, hq.HQ_RMS_Y):
                o = hq.rms_norm(hq.RmsNormDesc(C, 1e-6, outputs, dt, hq.F32), x, gamma, r)
                _, y, codes, scales = rms64(x, r, gamma, 1e-6)
                # h itself carries one rounding of the sum, of |x + r|
                assert_within(o.y, y, 28 * U32 * y.abs() + 1e-30, f"T={T} C={C} y")
                if o.scales is not None:
                    assert_within(o.scales[:, None], scales[:, None], 30 * U32 * scales[:, None], f"T={T} C={C} scales")
                    assert torch.equal(o.codes, codes)
