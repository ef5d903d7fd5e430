"""Host-side checks of the rotary positions: descriptors, frequencies and refusals
before anything is enqueued. No kernels run."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from hadamard_rotated_bit_amd import _lib

lib = _lib.load()
P = ctypes.c_void_p


def ref(q=4, k=2, dim=64, pairs=(8, 24), axes=None, layout=0, norm=0, inverse=0, pos=0, x=1, y=1, eps=1e-6):
    arr = (ctypes.c_int32 * 4)(*pairs)
    return ctypes.byref(_lib.HqRopeDesc(q, k, dim, len(pairs) if axes is None else axes, arr, layout, norm, inverse, pos, x, y, eps))


@pytest.mark.parametrize("kw,status", [
    (dict(q=-1), -1), (dict(k=-1), -1), (dict(dim=0), -1), (dict(axes=0), -1), (dict(axes=5), -1), (dict(pairs=(-4, 8)), -1),
    (dict(pairs=(1 << 30, 1 << 30)), -1), (dict(layout=2), -1), (dict(layout=-1), -1), (dict(norm=2), -1), (dict(inverse=-1), -1),
    (dict(pos=2), -1), (dict(x=2), -1), (dict(y=-1), -1), (dict(norm=1, eps=0.0), -1), (dict(norm=1, eps=float("nan")), -1),
    (dict(norm=1, eps=1e-31), -2), (dict(norm=1, inverse=1), -2), (dict(q=0, k=0), -2), (dict(q=1025), -2), (dict(q=1000, k=25), -2),
    (dict(q=2 ** 31 - 1, k=2 ** 31 - 1), -2), (dict(dim=60), -2), (dict(dim=264), -2), (dict(pairs=(8, 28)), -2),
    (dict(pairs=(8, 6)), -2), (dict(pairs=(0, 0)), -2)])
def test_descriptor_refusals(kw, status):
    assert lib.hq_rope_validate(ref(**kw)) == status
    assert len(lib.hq_last_error()) > 0


@pytest.mark.parametrize("kw", [dict(), dict(pairs=(3, 5)), dict(pairs=(0, 4, 0, 0)), dict(dim=8, pairs=(4,)), dict(dim=256, pairs=(128,)),
                                dict(q=0, k=1), dict(q=1024, k=0), dict(norm=1), dict(norm=1, eps=2.0 ** -100), dict(eps=0.0), dict(inverse=1), dict(dim=72, pairs=(18, 18))])
def test_descriptor_accepts(kw):
    assert lib.hq_rope_validate(ref(**kw)) == 0


def call(d=None, X=0x1000000, ldx=512, pos=0x10000, freqs=0x20000, gq=None, gk=None, T=100, Y=0x2000000, ldy=384):
    v = lambda p: None if p is None else P(p)
    return lib.hq_rope(d or ref(), v(X), ldx, v(pos), v(freqs), v(gq), v(gk), T, v(Y), ldy, None)


# pointers that are never dereferenced: every call below fails validation first
@pytest.mark.parametrize("kw,status,word", [
    (dict(X=None), -1, b"non-NULL"), (dict(pos=None), -1, b"non-NULL"), (dict(freqs=None), -1, b"non-NULL"),
    (dict(Y=None), -1, b"non-NULL"), (dict(T=-1), -1, b"T must"), (dict(T=(1 << 26) + 1), -2, b"at most"),
    (dict(ldx=376), -1, b"ldx"), (dict(ldy=376), -1, b"ldx"), (dict(ldx=516), -1, b"ldx"), (dict(ldy=388), -1, b"ldx"),
    (dict(ldx=-512), -1, b"ldx"), (dict(ldx=1 << 40), -1, b"ldx"),
    (dict(X=0x1000008), -1, b"aligned"), (dict(Y=0x2000004), -1, b"aligned"), (dict(freqs=0x20008), -1, b"aligned"),
    (dict(pos=0x10002), -1, b"aligned"), (dict(d=ref(norm=1), gq=0x1008), -1, b"aligned"), (dict(d=ref(norm=1), gk=0x1004), -1, b"aligned"),
    (dict(gq=0x1000), -1, b"without norm"), (dict(gk=0x1000), -1, b"without norm"),
    (dict(Y=0x1000000), -1, b"overlaps X"), (dict(Y=0x1000000, ldy=512, d=ref(y=0)), -1, b"overlaps X"),
    (dict(Y=0x1000000 + 512, ldy=512), -1, b"overlaps X"), (dict(pos=0x2000000), -1, b"overlaps positions"),
    (dict(freqs=0x2000010), -1, b"overlaps positions"), (dict(d=ref(norm=1), gq=0x2000000), -1, b"a gamma"),
    (dict(d=ref(norm=1), gk=0x2000010), -1, b"a gamma"),
])
def test_call_refusals(kw, status, word):
    assert call(**kw) == status
    assert word in lib.hq_last_error()


def test_empty_call_is_a_no_op():
    assert call(T=0, X=None, pos=None, freqs=None, Y=None) == 0


def test_frequencies():
    d = hq.RopeDesc(2, 1, 32, (3, 0, 5))
    f = hq.rope_freqs(d, 100.0, device="cpu")
    want = [100.0 ** (-i / 3) for i in range(3)] + [100.0 ** (-i / 5) for i in range(5)]
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=1e-15)
    f = hq.rope_freqs(d, 100.0, per_axis=False, device="cpu")
    assert torch.allclose(f, torch.tensor([100.0 ** (-i / 8) for i in range(8)], dtype=torch.float64), rtol=1e-15)


def test_python_refusals():
    with pytest.raises(ValueError, match="axes"):
        hq.RopeDesc(1, 1, 64, (4, 4, 4, 4, 4))
    with pytest.raises(ValueError, match="axes"):
        hq.RopeDesc(1, 1, 64, ())
    d = hq.RopeDesc(1, 1, 64, (32,))
    f = hq.rope_freqs(d, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        hq.rope(d, torch.zeros(3, 128), torch.zeros(3, 1, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="channels"):
        hq.rope(d, torch.zeros(3, 2, 64), torch.zeros(3, 1, dtype=torch.int32), f)
