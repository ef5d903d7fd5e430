"""Host-side checks of the RMS norm: descriptors and refusals before anything is
enqueued. No kernels run."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from hadamard_rotated_bit_amd import _lib

lib = _lib.load()
P = ctypes.c_void_p


def ref(channels=256, outputs=7, x_dtype=1, y_dtype=1, eps=1e-6):
    return ctypes.byref(_lib.HqRmsDesc(channels, outputs, x_dtype, y_dtype, eps))


@pytest.mark.parametrize("kw,status", [
    (dict(channels=0), -1), (dict(channels=-8), -1), (dict(outputs=0), -1), (dict(outputs=8), -1), (dict(outputs=-1), -1),
    (dict(x_dtype=2), -1), (dict(y_dtype=-1), -1), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(eps=1e-31), -2), (dict(eps=1e-44), -2), (dict(channels=252), -2), (dict(channels=8200), -2)])
def test_descriptor_refusals(kw, status):
    assert lib.hq_rms_validate(ref(**kw)) == status
    assert len(lib.hq_last_error()) > 0


def test_no_descriptor():
    assert lib.hq_rms_validate(None) == -1
    assert lib.hq_rms_norm(None, None, None, None, 0, None, None, None, None, None) == -1


@pytest.mark.parametrize("kw", [dict(), dict(channels=8), dict(channels=8192), dict(outputs=1), dict(eps=2.0 ** -100), dict(x_dtype=0, y_dtype=1)])
def test_descriptor_accepts(kw):
    assert lib.hq_rms_validate(ref(**kw)) == 0


def call(d=None, X=0x100000, r=0x200000, gamma=0x1000, T=100, H=0x300000, Y=0x400000, codes=0x500000, scales=0x600000):
    v = lambda p: None if p is None else P(p)
    return lib.hq_rms_norm(d or ref(), v(X), v(r), v(gamma), T, v(H), v(Y), v(codes), v(scales), None)


# pointers that are never dereferenced: every call below fails validation first
@pytest.mark.parametrize("kw,status,word", [
    (dict(X=None), -1, b"non-NULL"), (dict(H=None), -1, b"non-NULL"), (dict(Y=None), -1, b"non-NULL"),
    (dict(codes=None), -1, b"non-NULL"), (dict(scales=None), -1, b"non-NULL"),
    (dict(T=-1), -1, b"T must be"), (dict(T=(1 << 26) + 1), -2, b"at most"),
    (dict(X=0x100008), -1, b"aligned"), (dict(r=0x200004), -1, b"aligned"), (dict(gamma=0x1004), -1, b"aligned"),
    (dict(H=0x300002), -1, b"aligned"), (dict(Y=0x400008), -1, b"aligned"), (dict(codes=0x500001), -1, b"aligned"),
    (dict(scales=0x600004), -1, b"aligned"),
    (dict(H=0x100000 + 512), -1, b"H overlaps"), (dict(H=0x200000 + 512), -1, b"H overlaps"), (dict(H=0xff0), -1, b"H overlaps"),
    (dict(Y=0x100000 + 512), -1, b"Y overlaps"), (dict(Y=0x100000, d=ref(y_dtype=0)), -1, b"Y overlaps"),
    (dict(Y=0x1000), -1, b"Y overlaps"), (dict(codes=0x100000), -1, b"codes or scales"),
    (dict(codes=0x200000), -1, b"codes or scales"), (dict(scales=0x1010), -1, b"codes or scales"),
    (dict(H=0x400000), -1, b"each other"), (dict(codes=0x300010), -1, b"each other"), (dict(scales=0x400010), -1, b"each other"),
    (dict(codes=0x600000), -1, b"each other"), (dict(X=0x300000, Y=0x300000, H=0x300000), -1, b"each other"),
])
def test_call_refusals(kw, status, word):
    assert call(**kw) == status
    assert word in lib.hq_last_error()


def test_empty_call_is_a_no_op():
    assert call(T=0, X=None, H=None, Y=None, codes=None, scales=None) == 0


def test_python_refusals():
    d = hq.RmsNormDesc(64)
    with pytest.raises(ValueError, match="channels"):
        hq.rms_norm(d, torch.zeros(4, 4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        hq.rms_norm(d, torch.zeros(4, 64))
