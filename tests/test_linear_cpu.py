"""Host-side checks of the dense layer and its epilogue: descriptors,
workspaces and every refusal, before anything is enqueued. No kernels run."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from hadamard_rotated_bit_amd import _lib

lib = _lib.load()
P = ctypes.c_void_p


def ref(**kw):
    d = dict(d_in=1152, d_out=4608, x_dtype=1, w_dtype=1, y_dtype=1)
    d.update(kw)
    return ctypes.byref(_lib.HqLinearDesc(*[d[k] for k in ["d_in", "d_out", "x_dtype", "w_dtype", "y_dtype"]]))


@pytest.mark.parametrize("kw,status", [
    (dict(d_in=0), -1), (dict(d_out=-8), -1), (dict(x_dtype=2), -1), (dict(w_dtype=-1), -1),
    (dict(y_dtype=7), -1), (dict(x_dtype=0), -2), (dict(d_in=12), -2), (dict(d_out=4), -2),
    (dict(d_in=65544), -2), (dict(d_out=65544), -2)])
def test_descriptor_refusals(kw, status):
    assert lib.hq_linear_validate(ref(**kw)) == status
    assert len(lib.hq_last_error()) > 0
    assert lib.hq_linear_workspace_bytes(ref(**kw), 100) == 0


def test_null_descriptor():
    assert lib.hq_linear_validate(None) == -1
    assert lib.hq_linear(None, P(0x1000), P(0x1000), None, 1, None, P(0x1000), None, 0, None) == -1


@pytest.mark.parametrize("kw", [dict(), dict(y_dtype=0), dict(x_dtype=0, w_dtype=0), dict(d_in=8, d_out=8),
                                dict(d_in=65536, d_out=65536)])
def test_descriptor_accepts(kw):
    assert lib.hq_linear_validate(ref(**kw)) == 0


def test_workspace_only_for_split_products():
    assert lib.hq_linear_workspace_bytes(ref(), 8192) == 0       # tiles for every CU
    assert lib.hq_linear_workspace_bytes(ref(), 1) == 0          # vector kernel
    assert lib.hq_linear_workspace_bytes(ref(), 0) == 0
    n = lib.hq_linear_workspace_bytes(ref(d_in=4096, d_out=1152), 100)
    assert n > 0 and n % (100 * 1152 * 4) < 256                  # whole partial matrices
    assert lib.hq_linear_workspace_bytes(ref(), -1) == 0
    with pytest.raises(hq.HqError):
        hq.linear_workspace_bytes(hq.LinearDesc(64, 64), -1)
    with pytest.raises(hq.HqError):
        hq.linear_workspace_bytes(hq.LinearDesc(63, 64), 1)


def call(d=None, X=0x10000, W=0x20000000, b=None, T=16, epi=None, Y=0x40000000, ws=None, n=0):
    e = ctypes.byref(epi) if epi is not None else None
    v = lambda p: None if p is None else P(p)
    return lib.hq_linear(d or ref(), v(X), v(W), v(b), T, e, v(Y), v(ws), n, None)


def epi(act=0, residual=None, gate=None, gate_rows=0, gate_ld=0):
    return _lib.HqEpilogue(act, residual, gate, gate_rows, gate_ld)


# pointers that are never dereferenced: every call below fails validation first
@pytest.mark.parametrize("kw,status,word", [
    (dict(X=None), -1, b"non-NULL"), (dict(W=None), -1, b"non-NULL"), (dict(Y=None), -1, b"non-NULL"),
    (dict(T=-1), -1, b"T must be"), (dict(T=(1 << 26) + 1), -2, b"T must be"),
    (dict(X=0x10008), -1, b"aligned"), (dict(W=0x20000004), -1, b"aligned"), (dict(b=0x3008), -1, b"aligned"),
    (dict(Y=0x40000002), -1, b"aligned"), (dict(ws=0x5001), -1, b"aligned"),
    (dict(Y=0x10000), -1, b"overlaps"), (dict(Y=0x10000 + 16 * 1152 * 2 - 16), -1, b"overlaps"),
    (dict(Y=0x20000000 + 4096), -1, b"overlaps"), (dict(b=0x40000000), -1, b"overlaps"),
    (dict(epi=epi(act=5)), -1, b"hq_act"), (dict(epi=epi(act=-1)), -1, b"hq_act"),
    (dict(epi=epi(residual=0x8)), -1, b"aligned"), (dict(epi=epi(gate=0x8, gate_rows=1, gate_ld=4608)), -1, b"aligned"),
    (dict(epi=epi(gate=0x5000, gate_ld=4608)), -1, b"gate_rows"),
    (dict(epi=epi(gate=0x5000, gate_rows=-3, gate_ld=4608)), -1, b"gate_rows"),
    (dict(epi=epi(gate=0x5000, gate_rows=4, gate_ld=4600)), -1, b"gate_ld"),
    (dict(epi=epi(gate=0x5000, gate_rows=4, gate_ld=4612)), -1, b"gate_ld"),
    (dict(epi=epi(gate=0x40000000, gate_rows=4, gate_ld=4608)), -1, b"gate overlaps"),
    (dict(epi=epi(residual=0x40000000 + 9216)), -1, b"residual overlaps"),
])
def test_call_refusals(kw, status, word):
    assert call(**kw) == status
    assert word in lib.hq_last_error()


def test_workspace_refused_when_missing_or_small():
    d = ref(d_in=4096, d_out=1152)
    n = lib.hq_linear_workspace_bytes(d, 100)
    assert call(d=d, T=100) == -3
    assert call(d=d, T=100, ws=0x5000, n=n - 1) == -3
    assert b"workspace" in lib.hq_last_error()
    # X, weight and Y of this call are at 0x10000, 0x20000000 and 0x40000000
    for at in (0x10000, 0x20000000 + 4096, 0x40000000 - 16):
        assert call(d=d, T=100, ws=at, n=n) == -1
        assert b"workspace overlaps" in lib.hq_last_error()
    for e in (epi(residual=0x5000), epi(gate=0x5000, gate_rows=8, gate_ld=1152)):
        assert call(d=d, T=100, ws=0x5000, n=n, epi=e) == -1
        assert b"workspace overlaps" in lib.hq_last_error()


def test_empty_call_is_a_no_op():
    assert call(T=0, X=None, W=None, Y=None) == 0


def test_python_refusals():
    d = hq.LinearDesc(64, 32)
    X = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        hq.linear(d, X, torch.zeros(32, 64))
    with pytest.raises(ValueError, match="residual"):
        hq.Epilogue(residual=torch.zeros(4, 32))._c(4, 32, torch.float32, 0)
    with pytest.raises(ValueError, match="gate"):
        hq.Epilogue(gate=torch.zeros(1, 32), gate_rows=4)._c(4, 32, torch.float32, 0)
