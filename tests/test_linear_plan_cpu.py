"""hq_linear's choice of a kernel, on the host: the GPU tests' shapes run the kernels that
they name, and they name every one that any size runs. No kernels run."""
import itertools

import pytest

import hadamard_rotated_bit_amd as hq
from test_gpu_linear_kernels import KERNELS, rows_form


def key(dt, T, K, N):
    p = hq.linear_plan(hq.LinearDesc(K, N, dt, dt, dt), T)
    return dt, p.kernel, p.splits > 1, rows_form(T, N) if p.kernel == hq.HQ_LINEAR_ROWS else None


@pytest.mark.parametrize("want", list(KERNELS))
def test_shapes_run_the_kernel_they_are_listed_for(want):
    T, N, Ks = KERNELS[want]
    for K in Ks:
        assert key(want[0], T, K, N) == want, (T, K, N)


def test_every_kernel_is_listed():
    T = [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65] + [int(100 * 1.35 ** e) for e in range(22)]
    N = [8, 16, 64, 72, 128, 136, 256] + [int(50 * 1.4 ** e) * 8 for e in range(15)]
    K = [8, 64, 72, 256, 328, 520, 776, 1160, 1544, 2056, 3080, 4104, 8200]
    found = {key(dt, t, k, n) for dt in (hq.F32, hq.BF16) for t, n, k in itertools.product(T, N, K)}
    assert found == set(KERNELS)


def test_plan_of_nothing_and_refusals():
    d = hq.LinearDesc(64, 32)
    p = hq.linear_plan(d, 0)
    assert (p.kernel, p.splits) == (0, 0)
    with pytest.raises(hq.HqError):
        hq.linear_plan(d, -1)
    with pytest.raises(hq.HqError):
        hq.linear_plan(hq.LinearDesc(63, 32), 1)
    assert hq.load().hq_linear_plan_of(d._ref, 1, None) == -1


def test_a_split_has_a_workspace_and_nothing_else_has():
    for dt, T, K, N in itertools.product((hq.F32, hq.BF16), (1, 33, 100, 250, 1000, 8200), (8, 1160, 4104), (136, 1160, 4104)):
        d = hq.LinearDesc(K, N, dt, dt, dt)
        n, s = hq.linear_workspace_bytes(d, T), hq.linear_plan(d, T).splits
        assert n == (0 if s == 1 else -(-s * T * N * 4 // 256) * 256)
