"""hq_adapters in tiles of rows against float64: every activation, gate and residual under
ranks of one k-step to eight, every pair of types, rows in runs and mixed, in place on base
and on the residual, one slab of columns and several, u in one part and in several. The
references and tolerances are those of test_gpu_adapters.py."""
import pytest

import hadamard_rotated_bit_amd as hq
from epilogue_ref import ACTS
from test_gpu_adapters import in_tiles, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("r", [16, 40, 72, 128])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("ydt", [hq.BF16, hq.F32])
def test_epilogues_at_every_rank(act, r, dt, ydt):
    T = 2100
    assert in_tiles(T, 72, 200, r, dt)
    for kind in ("runs", "mixed"):
        run(T, 72, 200, r, 5, dt, ydt, kind, act=act)
        run(T, 72, 200, r, 5, dt, ydt, kind, act=act, residual=True, gate_rows=T // 3 + 1)
        run(T, 72, 200, r, 5, dt, ydt, kind, act=act, residual=True, inplace="residual")
        run(T, 72, 200, r, 5, dt, ydt, kind, act=act, gate_rows=1, inplace="base")
        run(T, 72, 200, r, 5, dt, ydt, kind, act=act, scaled=False, based=False)
        run(T, 72, 200, r, 5, dt, ydt, kind, act=act, inplace="base")


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("r", [24, 64, 96])
def test_many_slabs_and_parts(act, r, dt):
    # 17 slabs in groups of two; K long enough for u in several parts
    for T, K in ((2049, 4104), (5000, 264)):
        assert in_tiles(T, K, 2120, r, dt)
        run(T, K, 2120, r, 4, dt, act=act, kind="mixed")
        run(T, K, 2120, r, 4, dt, act=act, residual=True, gate_rows=700, inplace="base")


@pytest.mark.parametrize("r", [8, 32, 64, 128])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("ydt", [hq.BF16, hq.F32])
def test_row_by_row_at_every_rank(r, dt, ydt):
    for act in ACTS:
        for T, kind in ((1, "one"), (24, "mixed"), (260, "mixed")):
            assert not in_tiles(T, 72, 200, r, dt)
            run(T, 72, 200, r, 9, dt, ydt, kind, act=act, residual=True, gate_rows=T // 3 + 1, inplace="base")
            run(T, 72, 200, r, 9, dt, ydt, kind, act=act, residual=True, inplace="residual")
