"""The activations of the dense layer's epilogue against float64, within what include/hq.h
states: for fp32 results 16 U (V >= 0) and 8 U (1 + |V| (1 + V^2 / 10)) (V < 0), relative, U =
2^-24, and 2^-119 absolute. Where that comes from: the exponent's argument a is good to two
(SiLU: the constant, the product), five (tanh form: x^2, two constants, the fused sum, the
product) or three (GELU: two products, the constant) roundings, |a| U ln 2 each of e^a; exp2,
the reciprocal and the last product add 6 U, GELU's fit 0.3 U and its ten steps 3 U.
|a| ln 2 is |V|, 1.6 |V| (1 + V^2 / 22) and V^2 / 2. The reciprocal of 1 + e^a above 2^126
would be a subnormal and is 0 instead: there |phi| <= |V| 2^-126, and V >= -87.4 = -126 ln 2,
above -2^7, in SiLU (closer to 0 in the others), or the value is smaller still: 2^-119."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import ACTS, U32, phi64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("lo,hi", [(-90, -10), (-10, -3), (-3, -0.5), (-0.5, -1e-6), (1e-6, 0.5), (0.5, 5), (5, 100)])
def test_fp32_results(lo, hi, act):
    # V itself is exact: x times 1 in a row of zeros
    v = torch.linspace(lo, hi, 1 << 20, device="cuda")
    X, W = torch.zeros(v.numel(), 8, device="cuda"), torch.zeros(8, 8, device="cuda")
    X[:, 0], W[:, 0] = v, 1.0
    Y = hq.linear(hq.LinearDesc(8, 8), X, W, epilogue=hq.Epilogue(ACTS[act]))
    assert torch.equal(hq.linear(hq.LinearDesc(8, 8), X, W)[:, 3], v)
    y, d = phi64(v, act), v.double()
    units = 16.0 if lo > 0 else 8.0 * (1.0 + d.abs() * (1.0 + d * d / 10.0))
    over = (Y - y[:, None]).abs() - (units * U32 * y.abs() + 2.0 ** -119)[:, None]
    assert not bool((over > 0).any()), f"worst {((Y - y[:, None]).abs() / y[:, None].abs()).max().item() / U32:.1f} U"
