"""Host-side checks of the group norm: descriptors, workspaces and refusals
before anything is enqueued. No kernels run."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from hadamard_rotated_bit_amd import _lib

lib = _lib.load()
P = ctypes.c_void_p


def ref(channels=256, groups=32, act=0, x_dtype=1, y_dtype=1, eps=1e-5):
    return ctypes.byref(_lib.HqNormDesc(channels, groups, act, x_dtype, y_dtype, eps))


@pytest.mark.parametrize("kw,status", [
    (dict(channels=0), -1), (dict(groups=0), -1), (dict(groups=-4), -1), (dict(act=5), -1), (dict(act=-1), -1),
    (dict(x_dtype=2), -1), (dict(y_dtype=-1), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(channels=252, groups=4), -2), (dict(channels=4104, groups=1), -2),
    (dict(groups=48), -2), (dict(groups=512), -2)])
def test_descriptor_refusals(kw, status):
    assert lib.hq_norm_validate(ref(**kw)) == status
    assert len(lib.hq_last_error()) > 0
    assert lib.hq_group_norm_workspace_bytes(ref(**kw), 1, 1 << 20) == 0


@pytest.mark.parametrize("kw", [dict(), dict(channels=320), dict(channels=8, groups=8), dict(channels=4096, groups=1),
                                dict(channels=4096, groups=4096), dict(eps=0.0), dict(x_dtype=0, y_dtype=1)])
def test_descriptor_accepts(kw):
    assert lib.hq_norm_validate(ref(**kw)) == 0


def call(d=None, X=0x100000, gamma=None, beta=None, S=2, Pn=100, Y=0x40000000, ws=None, n=0):
    v = lambda p: None if p is None else P(p)
    return lib.hq_group_norm(d or ref(), v(X), v(gamma), v(beta), S, Pn, v(Y), v(ws), n, None)


# pointers that are never dereferenced: every call below fails validation first
@pytest.mark.parametrize("kw,status,word", [
    (dict(X=None), -1, b"non-NULL"), (dict(Y=None), -1, b"non-NULL"),
    (dict(S=-1), -1, b"samples"), (dict(Pn=-1), -1, b"samples"),
    (dict(S=1 << 20, Pn=1 << 20), -2, b"at most"), (dict(S=(1 << 26) + 1, Pn=1), -2, b"at most"),
    (dict(S=1 << 62, Pn=4), -2, b"at most"),
    (dict(X=0x100008), -1, b"aligned"), (dict(Y=0x40000004), -1, b"aligned"), (dict(gamma=0x1004), -1, b"aligned"),
    (dict(beta=0x1008), -1, b"aligned"), (dict(ws=0x1008), -1, b"aligned"),
    (dict(Y=0x100000 + 512), -1, b"overlaps X"), (dict(Y=0x100000, d=ref(y_dtype=0)), -1, b"overlaps X"),
    (dict(gamma=0x40000000), -1, b"overlaps gamma"), (dict(beta=0x40000400), -1, b"overlaps gamma or beta"),
])
def test_call_refusals(kw, status, word):
    assert call(**kw) == status
    assert word in lib.hq_last_error()


def test_workspace():
    d = ref(channels=128)
    n = lib.hq_group_norm_workspace_bytes(d, 1, 262144)
    assert n >= 8 * 32
    assert lib.hq_group_norm_workspace_bytes(d, 4, 0) == 0 and lib.hq_group_norm_workspace_bytes(d, -1, 5) == 0
    assert lib.hq_group_norm_workspace_bytes(ref(channels=1152, groups=1), 8192, 1) == 0   # one launch
    big = dict(d=d, S=1, Pn=262144, X=0x100000, Y=0x40000000)
    assert call(**big) == -3
    assert call(**big, ws=0x5000, n=n - 1) == -3
    assert b"workspace" in lib.hq_last_error()
    for at in (0x100000, 0x40000000 - 16):
        assert call(**big, ws=at, n=n) == -1
        assert b"workspace overlaps" in lib.hq_last_error()


def test_empty_calls_are_no_ops():
    assert call(S=0, X=None, Y=None) == 0
    assert call(Pn=0, X=None, Y=None) == 0


def test_python_refusals():
    d = hq.NormDesc(64, 8)
    with pytest.raises(ValueError, match="positions"):
        hq.group_norm(d, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        hq.group_norm(d, torch.zeros(1, 4, 64))
    with pytest.raises(hq.HqError):
        hq.group_norm_workspace_bytes(d, -1, 4)
    with pytest.raises(hq.HqError):
        hq.group_norm_workspace_bytes(hq.NormDesc(64, 7), 1, 4)
