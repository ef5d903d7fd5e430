"""Host-side checks of the adapters: descriptors, workspaces and refusals before
anything is enqueued. No kernels run."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from hadamard_rotated_bit_amd import _lib

lib = _lib.load()
P = ctypes.c_void_p


def ref(d_in=256, d_out=512, rank=16, x=1, w=1, y=1):
    return ctypes.byref(_lib.HqAdapterDesc(d_in, d_out, rank, x, w, y))


BAD = [(dict(d_in=0), -1), (dict(d_out=-8), -1), (dict(x=2), -1), (dict(w=-1), -1), (dict(y=2), -1), (dict(x=0), -2),
       (dict(d_in=252), -2), (dict(d_out=12), -2), (dict(d_in=65544), -2), (dict(d_out=65544), -2), (dict(rank=0), -2),
       (dict(rank=-8), -2), (dict(rank=12), -2), (dict(rank=136), -2)]


@pytest.mark.parametrize("kw,status", BAD)
def test_descriptor_refusals(kw, status):
    assert lib.hq_adapter_validate(ref(**kw)) == status
    assert len(lib.hq_last_error()) > 0
    assert lib.hq_adapters_workspace_bytes(ref(**kw), 100) == 0


@pytest.mark.parametrize("kw", [dict(), dict(d_in=8, d_out=8, rank=8), dict(d_in=65536, d_out=65536, rank=128), dict(x=0, w=0), dict(y=0)])
def test_descriptor_accepts(kw):
    assert lib.hq_adapter_validate(ref(**kw)) == 0


def call(d=None, X=0x10000000, A=0x20000000, B=0x30000000, count=5, ids=0x1000, scales=0x8000, base=0x40000000, T=100, epi=None,
         Y=0x50000000, ws=0x60000000, n=1 << 30):
    v = lambda p: None if p is None else P(p)
    return lib.hq_adapters(d or ref(), v(X), v(A), v(B), count, v(ids), v(scales), v(base), T, epi, v(Y), v(ws), n, None)


def epi(act=0, residual=None, gate=None, rows=0, ld=0):
    return ctypes.byref(_lib.HqEpilogue(act, residual, gate, rows, ld))


# pointers that are never dereferenced: every call below fails validation first
@pytest.mark.parametrize("kw,status,word", [
    (dict(X=None), -1, b"non-NULL"), (dict(A=None), -1, b"non-NULL"), (dict(B=None), -1, b"non-NULL"),
    (dict(ids=None), -1, b"non-NULL"), (dict(Y=None), -1, b"non-NULL"), (dict(count=-1), -1, b"count"),
    (dict(T=-1), -1, b"T must"), (dict(T=(1 << 26) + 1), -2, b"at most"),
    (dict(X=0x10000008), -1, b"aligned"), (dict(A=0x20000002), -1, b"aligned"), (dict(B=0x30000004), -1, b"aligned"),
    (dict(ids=0x1002), -1, b"aligned"), (dict(scales=0x8004), -1, b"aligned"), (dict(base=0x40000008), -1, b"aligned"),
    (dict(Y=0x50000008), -1, b"aligned"), (dict(ws=0x60000008), -1, b"aligned"),
    (dict(Y=0x10000000), -1, b"Y overlaps"), (dict(Y=0x20000010), -1, b"Y overlaps"), (dict(Y=0x30000010), -1, b"Y overlaps"),
    (dict(Y=0xff0), -1, b"Y overlaps"), (dict(Y=0x8010), -1, b"Y overlaps"), (dict(Y=0x40000010), -1, b"Y overlaps"),
    (dict(epi=epi(act=7)), -1, b"act"), (dict(epi=epi(residual=0x50000010)), -1, b"residual overlaps"),
    (dict(epi=epi(gate=0x7000, rows=0, ld=512)), -1, b"gate_rows"), (dict(epi=epi(gate=0x7000, rows=10, ld=504)), -1, b"gate_ld"),
])
def test_call_refusals(kw, status, word):
    assert call(**kw) == status
    assert word in lib.hq_last_error()


def test_workspace():
    # rows one by one need none, tiles of rows a row's products with A for each part of K
    assert lib.hq_adapters_workspace_bytes(ref(), 100) == 0
    n = lib.hq_adapters_workspace_bytes(ref(), 5000)
    assert n >= 5000 * 16 * 4
    assert lib.hq_adapters_workspace_bytes(ref(), 0) == 0 and lib.hq_adapters_workspace_bytes(ref(), -1) == 0
    assert call(T=5000, ws=None, n=0) == -3
    assert call(T=5000, n=n - 1) == -3
    assert b"workspace" in lib.hq_last_error()
    for at in (0x10000000, 0x20000000, 0x30000010, 0x1000, 0x8000, 0x40000000, 0x50000000 - 16):
        assert call(T=5000, ws=at, n=n) == -1
        assert b"workspace overlaps" in lib.hq_last_error()


def test_workspace_over_the_range():
    # from one row to the most, every rank: never negative, never more than 256 parts
    for T in (1, 4, 5, 64, 256, 257, 2048, 2049, 8192, 100_000, 1 << 26):
        for d_in, d_out, rank in ((8, 8, 8), (65536, 8, 128), (8, 65536, 64), (65536, 65536, 128), (4096, 4096, 16)):
            for dt in (0, 1):
                n = lib.hq_adapters_workspace_bytes(ref(d_in, d_out, rank, dt, dt, dt), T)
                assert n == 0 or T * rank * 4 <= n <= 256 * T * rank * 4 + 256
                assert n > 0 or T <= 2048


def test_empty_call_is_a_no_op():
    assert call(T=0, X=None, A=None, B=None, ids=None, Y=None, ws=None, n=0) == 0


def test_python_refusals():
    d = hq.AdapterDesc(64, 64, 8)
    z = torch.zeros
    with pytest.raises(ValueError, match="d_in"):
        hq.adapters(d, z(2, 4, 64), z(1, 8, 64), z(1, 64, 8), z(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        hq.adapters(d, z(4, 64), z(1, 8, 64), z(1, 64, 8), z(4, dtype=torch.int32))
    with pytest.raises(hq.HqError):
        hq.adapters_workspace_bytes(d, -1)
    with pytest.raises(hq.HqError):
        hq.adapters_workspace_bytes(hq.AdapterDesc(64, 64, 12), 4)
