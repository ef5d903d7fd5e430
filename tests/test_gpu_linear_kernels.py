"""Every kernel that hq_linear chooses (hq.linear_plan), each under its own name: values
against float64 from one k-step to many, odd and even counts, chunks past the end of K and
tiles past the end on every side; the memory around the operands; two streams at once;
graph replays. test_linear_plan_cpu.py holds the list to the plan, so a shape whose kernel
changes fails there instead of leaving a kernel untested."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT, U32, assert_within
from test_gpu_linear import make, run

pytestmark = pytest.mark.gpu

BF, F = hq.BF16, hq.F32


def rows_form(T, N):
    """Rows and columns per wave of the vector kernel."""
    return (T if T <= 2 else 4), (2 if N >= 4096 else 1)


# (type, kernel, split, rows form): T, N and the d_in of its cases, the first for the memory, stream and graph tests
KERNELS = {
    (BF, hq.HQ_LINEAR_ROWS, False, (1, 1)): (1, 200, [328, 8, 2056, 4104]),
    (BF, hq.HQ_LINEAR_ROWS, False, (1, 2)): (1, 4104, [1160, 8, 2056, 4104]),
    (BF, hq.HQ_LINEAR_ROWS, False, (2, 1)): (2, 200, [328, 8, 2056, 4104]),
    (BF, hq.HQ_LINEAR_ROWS, False, (2, 2)): (2, 4104, [1160, 8, 2056]),
    (BF, hq.HQ_LINEAR_ROWS, False, (4, 1)): (3, 200, [1160, 1544, 4104]),
    (BF, hq.HQ_LINEAR_FEW, False, None): (40, 136, [328, 8, 64, 72, 520, 1544, 2056]),
    (BF, hq.HQ_LINEAR_T32, False, None): (300, 1160, [456, 8, 64, 136, 328, 1544]),
    (BF, hq.HQ_LINEAR_T32, True, None): (33, 1160, [4104, 4168, 6152]),
    (BF, hq.HQ_LINEAR_T32X4, False, None): (300, 1160, [2056, 2112, 2248, 4104]),
    (BF, hq.HQ_LINEAR_T64X2, False, None): (590, 1160, [456, 8, 64, 136, 328, 2056]),
    (BF, hq.HQ_LINEAR_T64X128, False, None): (1000, 1160, [456, 8, 64, 136, 328, 2056]),
    (BF, hq.HQ_LINEAR_T128, False, None): (1100, 2312, [456, 8, 64, 136, 328, 2056]),
    (BF, hq.HQ_LINEAR_T128X2, False, None): (2000, 1800, [3080, 3136, 3208, 4104]),
    (BF, hq.HQ_LINEAR_T128W8, False, None): (2500, 2312, [456, 8, 64, 136, 328, 1160]),
    (BF, hq.HQ_LINEAR_T128X192, False, None): (1100, 4040, [2056, 2112, 2120, 3080, 3144]),
    (BF, hq.HQ_LINEAR_256X192, False, None): (8200, 1160, [456, 8, 64, 72, 128, 136, 200, 256, 264, 320, 328, 392, 520, 584, 1152, 1160]),
    (BF, hq.HQ_LINEAR_256X256, False, None): (4000, 4040, [456, 8, 64, 72, 128, 136, 200, 256, 264, 320, 328, 392, 520, 584, 1152]),
    (F, hq.HQ_LINEAR_ROWS, False, (1, 1)): (1, 200, [328, 8, 2056]),
    (F, hq.HQ_LINEAR_ROWS, False, (1, 2)): (1, 4104, [1160, 8]),
    (F, hq.HQ_LINEAR_ROWS, False, (2, 1)): (2, 200, [328, 8, 2056]),
    (F, hq.HQ_LINEAR_ROWS, False, (2, 2)): (2, 4104, [1160, 8]),
    (F, hq.HQ_LINEAR_ROWS, False, (4, 1)): (3, 200, [328, 8, 2056]),
    (F, hq.HQ_LINEAR_ROWS, False, (4, 2)): (4, 4104, [1160, 8]),
    (F, hq.HQ_LINEAR_FEW, False, None): (40, 136, [328, 8, 32, 72, 520, 1528]),
    (F, hq.HQ_LINEAR_T32, False, None): (130, 1160, [328, 8, 40, 136, 360]),
    (F, hq.HQ_LINEAR_T32, True, None): (130, 1160, [1160, 776, 2056]),
    (F, hq.HQ_LINEAR_T64X2, False, None): (590, 1160, [328, 8, 32, 72, 136]),
    (F, hq.HQ_LINEAR_T64X2, True, None): (250, 1160, [1160, 776, 2056]),
    (F, hq.HQ_LINEAR_T64, False, None): (1100, 2312, [328, 8, 32, 72, 136]),
    (F, hq.HQ_LINEAR_T128, False, None): (2100, 2312, [328, 8, 32, 72, 1160]),
    (F, hq.HQ_LINEAR_T128, True, None): (1000, 1160, [1160, 1544, 2056]),
}
ONE = [pytest.param(k[0], T, Ks[0], N, id="-".join(map(str, k))) for k, (T, N, Ks) in KERNELS.items()]


@pytest.mark.parametrize("dt,T,K,N", [(k[0], T, K, N) for k, (T, N, Ks) in KERNELS.items() for K in Ks])
def test_values(dt, T, K, N):
    run(T, K, N, dt, act="gelu", residual=True, gate_rows=-(-T // 3))
    run(T, K, N, dt, inplace=True, residual=True, bias=False)


@pytest.mark.parametrize("dt,T,K,N", ONE)
def test_memory_around_the_operands(dt, T, K, N):
    X, W, b, _ = make(T, K, N, dt)
    pad = 4096
    nan = float("nan")
    bx = torch.full((T * K + 2 * pad,), nan, dtype=DT[dt], device="cuda")
    bw = torch.full((N * K + 2 * pad,), nan, dtype=DT[dt], device="cuda")
    by = torch.full((T * N + 2 * pad,), 77.0, dtype=DT[dt], device="cuda")
    x, w = bx[pad:pad + T * K].view(T, K), bw[pad:pad + N * K].view(N, K)
    y = by[pad:pad + T * N].view(T, N)
    x.copy_(X)
    w.copy_(W)
    desc = hq.LinearDesc(K, N, dt, dt, dt)
    n = hq.linear_workspace_bytes(desc, T)
    ws = torch.full((n + 2 * pad,), 77, dtype=torch.uint8, device="cuda")
    hq.linear(desc, x, w, b, out=y, workspace=ws[pad:pad + n] if n else None)
    assert torch.equal(y, hq.linear(desc, X, W, b))
    assert bool((by[:pad] == 77.0).all()) and bool((by[pad + T * N:] == 77.0).all())
    assert bool((ws[:pad] == 77).all()) and bool((ws[pad + n:] == 77).all())


@pytest.mark.parametrize("dt,T,K,N", ONE)
def test_two_streams_at_once(dt, T, K, N):
    desc = hq.LinearDesc(K, N, dt, dt, dt)
    Xa, W, b, _ = make(T, K, N, dt)
    Xb = make(T, K, N, dt, seed=1)[0]
    ref = [hq.linear(desc, x, W, b) for x in (Xa, Xb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for rep in range(4):
        for k, x in enumerate((Xa, Xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.linear(desc, x, W, b))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[k]) for k in range(2) for y in got[k])


@pytest.mark.parametrize("dt,T,K,N", ONE)
def test_graph_replays(dt, T, K, N):
    desc = hq.LinearDesc(K, N, dt, dt, dt)
    Xa, W, b, g = make(T, K, N, dt)
    Xb = make(T, K, N, dt, seed=1)[0]
    epi = hq.Epilogue(hq.HQ_ACT_SILU, torch.randn(T, N, generator=g, device="cuda").to(DT[dt]))
    Ya, Yb = (hq.linear(desc, x, W, b, epilogue=epi) for x in (Xa, Xb))
    n = hq.linear_workspace_bytes(desc, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    Xg, out = Xa.clone(), torch.empty_like(Ya)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hq.linear(desc, Xg, W, b, epilogue=epi, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.linear(desc, Xg, W, b, epilogue=epi, out=out, workspace=ws)
    for rep in range(4):
        Xg.copy_(Xa if rep % 2 == 0 else Xb)
        graph.replay()
        other = hq.linear(desc, Xb, W, b, epilogue=epi)
        torch.cuda.synchronize()
        assert torch.equal(out, Ya if rep % 2 == 0 else Yb), f"replay {rep}"
        assert torch.equal(other, Yb)
    del graph


@pytest.mark.parametrize("T", [1, 5, 40, 300, 2100])
@pytest.mark.parametrize("e", [-100, -109, -112, -118, -126, -130, -140, -149])
@pytest.mark.parametrize("small", ["X", "W"])
def test_smallest_fp32_operands(T, e, small):
    # one operand at 2^e, the other at 2^100: what a part of a split loses is less than
    # 2^-133 of the small operand and, below 2^-110, nothing else than that
    K, N = 264, 136
    g = torch.Generator(device="cuda")
    g.manual_seed(T - e)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").double()
    X, W = (r(T, K) * 2.0 ** (e if small == "X" else 100)).float(), (r(N, K) * 2.0 ** (e if small == "W" else 100)).float()
    x, w = X.double(), W.double()
    v = x @ w.t().contiguous()
    size = x.abs() @ w.abs().t().contiguous()
    lost = 2.0 ** -133 * (w.abs().sum(1)[None, :] if small == "X" else x.abs().sum(1)[:, None])
    tol = (K + 6 + 8) * U32 * (size + lost) + (lost if T > 4 else 0.0) + 2.0 ** -149
    assert_within(hq.linear(hq.LinearDesc(K, N), X, W), v, tol.expand_as(v), f"T={T} e={e} {small}")
