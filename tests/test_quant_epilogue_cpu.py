"""Host-side refusals of hq_quant_linear_epi before anything is enqueued."""
import ctypes

import pytest

from hadamard_rotated_bit_amd import BF16, Desc, _lib

lib = _lib.load()
P = ctypes.c_void_p


def call(desc=None, prep=0x1000, X=0x100000, T=16, epi=None, Y=0x40000000, ws=0x80000000, n=1 << 30):
    d = desc or Desc(1152, 4608, 128, 4, 4, 1, False, 0, BF16, BF16, BF16)
    v = lambda p: None if p is None else P(p)
    e = ctypes.byref(_lib.HqEpilogue(*epi)) if epi else None
    return lib.hq_quant_linear_epi(d._ref, v(prep), v(X), T, e, v(Y), v(ws), n, None)


# pointers that are never dereferenced: every call below fails validation first
@pytest.mark.parametrize("kw,status,word", [
    (dict(desc=Desc(1152, 4608, 128, 3)), -2, b"a_bits"), (dict(T=-1), -1, b"T must be"),
    (dict(T=(1 << 26) + 1), -2, b"T must be"), (dict(X=None), -1, b"non-NULL"), (dict(Y=None), -1, b"non-NULL"),
    (dict(prep=None), -1, b"non-NULL"), (dict(ws=None), -1, b"non-NULL"), (dict(n=10), -3, b"workspace"),
    (dict(X=0x100008), -1, b"aligned"), (dict(Y=0x100000), -1, b"overlaps X"),
    (dict(epi=(9, None, None, 0, 0)), -1, b"hq_act"), (dict(epi=(0, 0x18, None, 0, 0)), -1, b"aligned"),
    (dict(epi=(0, 0x40000010, None, 0, 0)), -1, b"residual overlaps"),
    (dict(epi=(0, None, 0x5000, 0, 4608)), -1, b"gate_rows"), (dict(epi=(0, None, 0x5000, 8, 4604)), -1, b"gate_ld"),
    (dict(epi=(0, None, 0x40000000, 8, 4608)), -1, b"gate overlaps"),
    (dict(ws=0x100000), -1, b"workspace overlaps"), (dict(ws=0x40000000 + 256), -1, b"workspace overlaps"),
    (dict(epi=(0, 0x80000100, None, 0, 0)), -1, b"workspace overlaps"),
    (dict(epi=(0, None, 0x80000100, 8, 4608)), -1, b"workspace overlaps"),
])
def test_refusals(kw, status, word):
    assert call(**kw) == status
    assert word in lib.hq_last_error()


def test_empty_call_is_a_no_op():
    assert call(T=0, X=None, Y=None, prep=None, ws=None, n=0) == 0


BLOB = lib.hq_prepared_bytes(Desc(1152, 4608, 128, 4, 4, 1, False, 0, BF16, BF16, BF16)._ref)


@pytest.mark.parametrize("kw", [dict(prep=0x40000000), dict(prep=0x40000000 - BLOB + 256), dict(prep=0x40000000 + 16 * 4608 * 2 - 256),
                                dict(prep=0x80000000), dict(prep=0x80000000 - BLOB + 256), dict(ws=0x1000 + BLOB - 256)])
def test_written_buffers_must_not_overlap_the_weights(kw):
    # Y at 0x40000000, the workspace at 0x80000000, the blob at 0x1000 where not given
    assert call(**kw) == -1
    assert b"overlaps prepared" in lib.hq_last_error()


def test_python_checks_the_weights():
    import torch

    import hadamard_rotated_bit_amd as hq
    d = Desc(1152, 4608, 128, 4, 4, 1, False, 0, BF16, BF16, BF16)
    blob = torch.zeros(BLOB, dtype=torch.uint8)
    hq._need_prepared(d, blob, -1)
    for bad, word in ((blob[:-1], "needed"), (torch.zeros(2 * BLOB, dtype=torch.uint8)[::2], "contiguous"), (None, "tensor")):
        with pytest.raises(ValueError, match=word):
            hq._need_prepared(d, bad, -1)
    with pytest.raises(ValueError, match="prepared is on"):
        hq._need_prepared(d, blob, 0)
