"""Every form of hq_group_norm (hq.group_norm_plan) at every width of the units that share a
group (gcd of the group's channels and 8): values, memory around the operands, two streams
at once and graph replays."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT
from test_gpu_norm import make, run

pytestmark = pytest.mark.gpu

ROWS, BLOCK, CHUNKS, JOINED = hq.HQ_NORM_ROWS, hq.HQ_NORM_BLOCK, hq.HQ_NORM_CHUNKS, hq.HQ_NORM_CHUNKS_JOINED
WIDTHS = {1: [(40, 8), (264, 8)], 2: [(80, 8), (720, 8)], 4: [(96, 8), (1056, 8)], 8: [(64, 4), (1152, 1), (4096, 2)]}
CASES = [pytest.param(kernel, S, P, C, G, id=f"{kernel}-{S}x{P}x{C}/{G}")
         for kernel, sizes in {BLOCK: [(3, 2), (5, 60), (64, 300)], CHUNKS: [(60, 5000)], JOINED: [(1, 30_011), (3, 9001)]}.items()
         for S, P in sizes for unit in WIDTHS for C, G in WIDTHS[unit]
         if not (kernel == BLOCK and P > 2 and C > 100) and not (kernel == CHUNKS and C > 1200)]
CASES += [pytest.param(ROWS, S, 1, C, G, id=f"{ROWS}-{S}x1x{C}/{G}") for S in (3, 3001) for C, G in ((8, 1), (1152, 1), (1152, 18), (4096, 1), (4096, 2))]


def form(S, P, C, G, dt):
    return hq.group_norm_plan(hq.NormDesc(C, G, x_dtype=dt, y_dtype=dt), S, P).kernel


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("kernel,S,P,C,G", CASES)
def test_values_and_memory(kernel, S, P, C, G, dt):
    assert form(S, P, C, G, dt) == kernel
    run(S, P, C, G, dt)
    run(S, P, C, G, dt, act="none", inplace=True)
    X, ga, be = make(S, P, C, dt)
    desc = hq.NormDesc(C, G, x_dtype=dt, y_dtype=dt)
    m, pad = X.numel(), 4096
    bx = torch.full((m + 2 * pad,), float("nan"), dtype=DT[dt], device="cuda")
    by = torch.full((m + 2 * pad,), 77.0, dtype=DT[dt], device="cuda")
    x, y = bx[pad:pad + m].view(S, P, C), by[pad:pad + m].view(S, P, C)
    x.copy_(X)
    n = hq.group_norm_workspace_bytes(desc, S, P)
    ws = torch.full((n + 2 * pad,), 77, dtype=torch.uint8, device="cuda")
    hq.group_norm(desc, x, ga, be, out=y, workspace=ws[pad:pad + n] if n else None)
    assert torch.equal(y, hq.group_norm(desc, X, ga, be))
    assert bool((by[:pad] == 77.0).all()) and bool((by[pad + m:] == 77.0).all())
    assert bool((ws[:pad] == 77).all()) and bool((ws[pad + n:] == 77).all())


@pytest.mark.parametrize("kernel,S,P,C,G", CASES)
def test_streams_and_graph_replays(kernel, S, P, C, G):
    dt = hq.BF16
    desc = hq.NormDesc(C, G, act=hq.HQ_ACT_SILU, x_dtype=dt, y_dtype=dt)
    Xa, ga, be = make(S, P, C, dt)
    Xb = make(S, P, C, dt, seed=5)[0]
    Ya, Yb = hq.group_norm(desc, Xa, ga, be), hq.group_norm(desc, Xb, ga, be)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for rep in range(3):
        for k, x in enumerate((Xa, Xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.group_norm(desc, x, ga, be))
    torch.cuda.synchronize()
    assert all(torch.equal(y, (Ya, Yb)[k]) for k in range(2) for y in got[k])
    n = hq.group_norm_workspace_bytes(desc, S, P)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    Xg, out = Xa.clone(), torch.empty_like(Xa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.group_norm(desc, Xg, ga, be, out=out, workspace=ws)
    for rep in range(4):
        Xg.copy_(Xa if rep % 2 == 0 else Xb)
        graph.replay()
        other = hq.group_norm(desc, Xb, ga, be)
        torch.cuda.synchronize()
        assert torch.equal(out, Ya if rep % 2 == 0 else Yb), f"replay {rep}"
        assert torch.equal(other, Yb)
    del graph
