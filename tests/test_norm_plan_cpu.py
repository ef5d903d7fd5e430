"""Host-side arithmetic of the group norm's launches over everything that the checks
accept: a grid holds less than 2^32 threads. No kernels run."""
import itertools

import pytest

import hadamard_rotated_bit_amd as hq
from test_gpu_norm_kernels import CASES, form

LIMIT = 1 << 26     # samples x positions


def near(n):
    return [v for v in (n - 1, n, n + 1) if v >= 1]


SAMPLES = sorted({v for e in range(0, 27, 2) for v in near(1 << e) if v <= LIMIT})
POSITIONS = sorted({v for n in (1, 2, 8, 16, 33, 64, 512, 2048, 1 << 15, 1 << 20, LIMIT) for v in near(n) if v <= LIMIT})


@pytest.mark.parametrize("dt", [hq.F32, hq.BF16])
@pytest.mark.parametrize("C,G", [(8, 1), (8, 8), (40, 4), (128, 32), (512, 16), (1024, 1), (1024, 1024), (2048, 32), (2056, 8),
                                 (4096, 1), (4096, 2), (4096, 32), (4096, 512), (4096, 4096)])
def test_every_grid_fits(C, G, dt):
    d = hq.NormDesc(C, G, x_dtype=dt, y_dtype=dt)
    for S, P in itertools.product(SAMPLES, POSITIONS):
        if S * P > LIMIT:
            continue
        p = hq.group_norm_plan(d, S, P)
        assert 0 < p.grid <= 1 << 31 and 1 <= p.slices <= S, (S, P, p.grid, p.slices)
        if p.slices > 1:        # no more launches than the threads ask for
            assert p.grid > 1 << 30, (S, P, p.grid, p.slices)


def test_forms():
    d = hq.NormDesc(1152, 1)
    p = hq.group_norm_plan(d, 8192, 1)
    assert (p.kernel, p.slices) == (hq.HQ_NORM_ROWS, 1)
    d = hq.NormDesc(512, 16, x_dtype=hq.BF16, y_dtype=hq.BF16)
    assert hq.group_norm_plan(d, 1 << 19, 33).slices == 1
    p = hq.group_norm_plan(d, 1 << 20, 33)      # 16 slabs of a block each: 2^32 threads in one launch
    assert (p.kernel, p.slices) == (hq.HQ_NORM_BLOCK, 2)
    d = hq.NormDesc(128, 32, x_dtype=hq.BF16, y_dtype=hq.BF16)
    assert hq.group_norm_plan(d, 1, 262144).kernel == hq.HQ_NORM_CHUNKS_JOINED
    assert hq.group_norm_plan(d, 64, 65536).kernel == hq.HQ_NORM_CHUNKS
    p = hq.group_norm_plan(d, 0, 5)
    assert (p.kernel, p.slices, p.grid) == (0, 0, 0)


def test_refusals():
    d = hq.NormDesc(64, 8)
    for S, P in ((-1, 4), (4, -1), (LIMIT, 2)):
        with pytest.raises(hq.HqError):
            hq.group_norm_plan(d, S, P)
    with pytest.raises(hq.HqError):
        hq.group_norm_plan(hq.NormDesc(64, 7), 1, 1)
    assert hq.load().hq_group_norm_plan(d._ref, 1, 1, None) == -1


@pytest.mark.parametrize("dt", [hq.F32, hq.BF16])
def test_gpu_shapes_run_the_form_they_are_listed_for(dt):
    for case in CASES:
        kernel, S, P, C, G = case.values
        assert form(S, P, C, G, dt) == kernel, case.id
    assert {c.values[0] for c in CASES} == {hq.HQ_NORM_ROWS, hq.HQ_NORM_BLOCK, hq.HQ_NORM_CHUNKS, hq.HQ_NORM_CHUNKS_JOINED}
