"""float64 reference of the epilogue Y = R + g phi(V) and the error a correct
fp32 implementation may have, element by element."""
import math

import torch

import hadamard_rotated_bit_amd as hq

ACTS = {"none": hq.HQ_ACT_NONE, "relu": hq.HQ_ACT_RELU, "silu": hq.HQ_ACT_SILU,
        "gelu": hq.HQ_ACT_GELU, "gelu_tanh": hq.HQ_ACT_GELU_TANH}
DT = {hq.F32: torch.float32, hq.BF16: torch.bfloat16}
U32 = 2.0 ** -24


def phi64(v, act):
    v = v.double()
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v / (1.0 + torch.exp(-math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def act_error(v, act, y_bf16):
    """Error of phi itself: the documented 1.1e-4 relative (1.5e-5 absolute
    beyond the fit) of the bf16 form of GELU; else the exponent's fp32
    rounding, 8 units of the argument |v| (1 + |v|^2 / 10), and 8 ulp."""
    p = phi64(v, act).abs()
    if act in ("none", "relu"):
        return torch.zeros_like(p)
    if act == "gelu" and y_bf16:
        return 1.1e-4 * p + 1.5e-5 * (v.abs() > 4.9)
    return 8 * U32 * p * (1.0 + v.abs() * (1.0 + v * v / 10.0)) + (1e-9 if y_bf16 else 0.0)


def epilogue64(v, v_err, act, y_dtype, residual=None, gate=None, gate_rows=0):
    """(y, tolerance) for the product v (float64, bias included) whose fp32
    value may be off by v_err. |phi'| <= 1.13 for every activation; each
    further fp32 operation adds half a unit of its result, and Y is rounded
    once to its type."""
    y = phi64(v, act)
    tol = 1.13 * v_err + act_error(v, act, y_dtype == hq.BF16)
    if gate is not None:
        g = gate.double()[torch.arange(v.shape[0], device=v.device) // gate_rows]
        y, tol = y * g, tol * g.abs() + U32 * (y * g).abs()
    if residual is not None:
        y = y + residual.double()
        tol = tol + U32 * y.abs()
    half = torch.finfo(DT[y_dtype]).eps / 2
    return y, tol * (1 + half) + half * y.abs() + 1e-30


def assert_within(got, y, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - y).abs() - tol)
    worst = over.max().item()
    assert worst <= 0, f"{what}: {int((over > 0).sum())} outside, worst by {worst:.3e} " \
                       f"at {divmod(int(over.argmax()), got.shape[-1])}"
