"""hq_linear against float64: every kernel variant and its borders (one row to
many, widths of one chunk and of ragged tiles, products split over d_in), the
epilogue's parts, in-place residuals, strided gates, non-finite rows, rows
behind the output, side streams and graph replays. Tolerances: K fp32
roundings of the absolute products (any order of sums), then epilogue_ref."""
import itertools

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import ACTS, DT, U32, assert_within, epilogue64

pytestmark = pytest.mark.gpu


def make(T, K, N, dt, seed=0, bias=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + T + 7 * K + 13 * N)
    X = torch.randn(T, K, generator=g, device="cuda").to(DT[dt])
    W = (torch.randn(N, K, generator=g, device="cuda") / K ** 0.5).to(DT[dt])
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    return X, W, b, g


def product64(X, W, b):
    x, w = X.double(), W.double()
    v = x @ w.t().contiguous()
    err = (X.shape[1] + 1) * U32 * (x.abs() @ w.abs().t().contiguous())
    if b is not None:
        v = v + b.double()
        err = err + U32 * v.abs()
    return v, err


def run(T, K, N, dt, ydt=None, act="none", residual=False, gate_rows=0, inplace=False, bias=True, seed=0):
    ydt = dt if ydt is None else ydt
    X, W, b, g = make(T, K, N, dt, seed, bias)
    R = torch.randn(T, N, generator=g, device="cuda").to(DT[ydt]) if residual else None
    G = None
    if gate_rows:
        table = torch.randn(-(-T // gate_rows), 3 * N, generator=g, device="cuda").to(DT[ydt])
        G = table[:, N:2 * N]      # one part of a modulation table
    v, err = product64(X, W, b)
    y, tol = epilogue64(v, err, act, ydt, R, G, gate_rows)
    desc = hq.LinearDesc(K, N, dt, dt, ydt)
    out = R if inplace else None
    epi = hq.Epilogue(ACTS[act], R, G, gate_rows)
    Y = hq.linear(desc, X, W, b, epilogue=epi, out=out)
    assert Y.dtype == DT[ydt] and (not inplace or Y.data_ptr() == R.data_ptr())
    assert_within(Y, y, tol, f"T={T} K={K} N={N} dt={dt} ydt={ydt} {act}")
    return Y


ROWS = [1, 2, 3, 4, 5, 8, 9, 31, 32, 33, 63, 65, 127, 129, 300]
WIDTHS = [(8, 8), (16, 24), (72, 136), (256, 1152), (1160, 264)]


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("K,N", WIDTHS)
def test_rows_and_widths(K, N, dt):
    for T in ROWS:
        run(T, K, N, dt)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,K,N", [(40, 4096, 64), (300, 4096, 1152), (130, 2056, 520), (17, 6144, 8),
                                   (2, 6144, 4104), (8, 8200, 4096)])
def test_long_sums(T, K, N, dt):
    # few output tiles: split over K, at a K that fills no k-step and no split evenly
    run(T, K, N, dt, act="silu", residual=True)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,K,N", [(2100, 1160, 2312), (4097, 256, 1096), (2049, 64, 4096), (5000, 24, 2304)])
def test_many_tiles(T, K, N, dt):
    run(T, K, N, dt, act="gelu", residual=True, gate_rows=-(-T // 3))


@pytest.mark.parametrize("K", [8, 64, 72, 128, 136, 192, 256, 320, 456, 1152])
@pytest.mark.parametrize("T,N", [(2500, 2312), (4000, 4040)])
def test_wide_tiles(T, N, K):
    # tiles of 256 x 192 and 256 x 256, from one k-step to many, odd and even counts, ragged on every side
    run(T, K, N, hq.BF16, act="gelu", residual=True, gate_rows=1000)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("K", [8, 64, 72, 136, 192, 328, 1096, 2056, 2248, 4104])
@pytest.mark.parametrize("T,N", [(9, 72), (100, 1160), (250, 1160), (590, 1160)])
def test_shared_k_steps(T, N, K, dt):
    # two and four groups of waves on a tile's k-steps: fewer steps than groups, odd and even counts, with and without a split
    run(T, K, N, dt, act="silu", residual=True, gate_rows=7)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,K,N", [(3, 8, 8), (17, 72, 40), (64, 256, 1160), (5, 4096, 4104), (8, 5128, 4096), (7, 264, 4104),
                                   (4000, 520, 8), (900, 1544, 24), (60, 776, 1160), (250, 3080, 256)])
def test_few_rows(T, K, N, dt):
    # k-steps shared by the waves of a block: fewer than waves, several rounds, chunks past the end of K
    run(T, K, N, dt, act="gelu", residual=True, gate_rows=2)
    run(T, K, N, dt, bias=False, inplace=True, residual=True)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,N", [(6724, 64), (12300, 8), (1100, 4040), (1100, 2312), (1000, 1160), (2050, 1160), (6001, 1000)])
@pytest.mark.parametrize("K", [8, 72, 328, 1544, 1608, 3208])
def test_middling_tiles(T, N, K, dt):
    # tiles of 128 x 192, 128 x 128 and 64 x 128, whole and split, from one k-step to many, ragged on every side
    run(T, K, N, dt, act="silu", residual=True, gate_rows=300)


@pytest.mark.parametrize("dt,ydt", list(itertools.product([hq.BF16, hq.F32], repeat=2)))
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T", [1, 7, 70, 700])
def test_epilogue_parts(T, act, dt, ydt):
    run(T, 328, 200, dt, ydt, act)
    run(T, 328, 200, dt, ydt, act, bias=False, residual=True)
    run(T, 328, 200, dt, ydt, act, gate_rows=1)
    run(T, 328, 200, dt, ydt, act, residual=True, gate_rows=max(1, T // 3), inplace=True)
    run(T, 328, 200, dt, ydt, act, residual=True, gate_rows=T + 5)


def test_empty_and_reused_output():
    desc = hq.LinearDesc(64, 32, hq.BF16, hq.BF16, hq.BF16)
    X, W, b, _ = make(5, 64, 32, hq.BF16)
    assert hq.linear(desc, X[:0].contiguous(), W, b).shape == (0, 32)
    out = torch.empty(5, 32, dtype=torch.bfloat16, device="cuda")
    assert hq.linear(desc, X, W, b, out=out) is out


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,K,N", [(3, 72, 40), (33, 72, 40), (300, 1032, 136), (2100, 520, 2312), (2500, 1032, 2312), (4000, 584, 4040)])
def test_neighbours_are_left_alone(T, K, N, dt):
    # the buffers around X, W and Y hold NaN and marks: no row, column or chunk
    # past the operands is read as data, nothing past Y is written
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
    hq.linear(desc, x, w, b, out=y)
    assert torch.equal(y, hq.linear(desc, X, W, b))
    assert bool((by[:pad] == 77.0).all()) and bool((by[pad + T * N:] == 77.0).all())


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T", [4, 40, 400])
def test_non_finite_rows_stay_in_their_rows(T, dt):
    X, W, b, _ = make(T, 328, 136, dt)
    desc = hq.LinearDesc(328, 136, dt, dt, dt)
    clean = hq.linear(desc, X, W, b, epilogue=hq.Epilogue(hq.HQ_ACT_SILU))
    X2 = X.clone()
    X2[1, 5], X2[3, 320] = float("nan"), float("inf")
    for act in ACTS.values():
        got = hq.linear(desc, X2, W, b, epilogue=hq.Epilogue(act))
        assert bool(torch.isnan(got[1]).all())
        assert not bool(torch.isfinite(got[3]).all())
        keep = [t for t in range(T) if t not in (1, 3)]
        if act == hq.HQ_ACT_SILU:
            assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("ydt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_range(act, ydt):
    # V runs over the whole fp32 range through a one-column weight of ones
    v = torch.cat([torch.linspace(-12, 12, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 3e38, -3e38])])
    v = torch.cat([v, -torch.logspace(-6, 2, 500), torch.logspace(-6, 2, 500)]).cuda()
    X = torch.zeros(v.numel(), 8, device="cuda")
    X[:, 0] = v
    W = torch.zeros(8, 8, device="cuda")
    W[:, 0] = 1.0
    Y = hq.linear(hq.LinearDesc(8, 8, hq.F32, hq.F32, ydt), X, W, epilogue=hq.Epilogue(ACTS[act]))
    y, tol = epilogue64(v.double()[:, None].expand(-1, 8), torch.zeros_like(v.double())[:, None], act, ydt)
    assert_within(Y, torch.nan_to_num(y, 0.0), tol.nan_to_num(1e-30), act)


@pytest.mark.parametrize("T", [4, 40, 2100])
def test_fp32_operands_of_every_size(T):
    # magnitudes from 1e-25 to near the largest float in one row of operands:
    # the parts of a split value are exact and no part overflows. Rows and
    # columns are scaled by powers of two, so the sums are those of plain data.
    K, N = 264, 136
    X, W, b, g = make(T, K, N, hq.F32, bias=False)
    ex = torch.randint(-40, 41, (T, 1), generator=g, device="cuda").double()
    ew = torch.randint(-40, 41, (N, 1), generator=g, device="cuda").double()
    X2, W2 = (X.double() * 2.0 ** ex).float(), (W.double() * 2.0 ** ew).float()
    Y = hq.linear(hq.LinearDesc(K, N, hq.F32, hq.F32, hq.F32), X2, W2)
    v, err = product64(X2, W2, None)
    assert_within(Y, *epilogue64(v, err, "none", hq.F32), "scaled rows")
    big = torch.finfo(torch.float32).max
    X3, W3 = torch.zeros(T, K, device="cuda"), torch.zeros(N, K, device="cuda")
    X3[:, 7], W3[:, 7] = big, 0.9990234375
    assert_within(hq.linear(hq.LinearDesc(K, N, hq.F32, hq.F32, hq.F32), X3, W3),
                  *epilogue64(*product64(X3, W3, None), "none", hq.F32), "largest")


@pytest.mark.parametrize("T,K,N", [(2, 1152, 6912), (300, 4096, 1152), (2500, 1160, 2312)])
def test_two_calls_at_once(T, K, N):
    # two streams, each with its own buffers, queued together
    desc = hq.LinearDesc(K, N, hq.BF16, hq.BF16, hq.BF16)
    Xa, W, b, g = make(T, K, N, hq.BF16)
    Xb = make(T, K, N, hq.BF16, seed=1)[0]
    ref = [hq.linear(desc, x, W, b) for x in (Xa, Xb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for rep in range(6):
        for k, x in enumerate((Xa, Xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.linear(desc, x, W, b))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[k]) for k in range(2) for y in got[k])


def test_offsets_past_32_bits():
    T, K, N = 270_001, 8192, 8   # X holds 2.2e9 values
    desc = hq.LinearDesc(K, N, hq.BF16, hq.BF16, hq.BF16)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    Xe, W, b, _ = make(64, K, N, hq.BF16)
    X[-64:] = Xe
    Y = hq.linear(desc, X, W, b)
    v, err = product64(Xe, W, b)
    assert_within(Y[-64:], *epilogue64(v, err, "none", hq.BF16), "last rows")
    assert torch.equal(Y[:1000], b.to(torch.bfloat16).expand(1000, N))


def test_side_stream_and_repeats():
    X, W, b, g = make(300, 4096, 1152, hq.BF16)
    desc = hq.LinearDesc(4096, 1152, hq.BF16, hq.BF16, hq.BF16)
    ref = hq.linear(desc, X, W, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [hq.linear(desc, X, W, b) for _ in range(5)]
    side.synchronize()
    assert all(torch.equal(ref, y) for y in got)


@pytest.mark.parametrize("T,K,N", [(2, 1152, 6912), (300, 4096, 1152), (2100, 1160, 2312), (4000, 584, 4040)])
def test_graph_replays_match_eager(T, K, N):
    desc = hq.LinearDesc(K, N, hq.BF16, hq.BF16, hq.BF16)
    Xa, W, b, g = make(T, K, N, hq.BF16)
    Xb = make(T, K, N, hq.BF16, seed=1)[0]
    R = torch.randn(T, N, generator=g, device="cuda").to(torch.bfloat16)
    epi = hq.Epilogue(hq.HQ_ACT_GELU_TANH, R)
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


@pytest.mark.parametrize("T", [1, 4, 7, 40, 300, 700, 2100])
@pytest.mark.parametrize("K,N", [(8, 1160), (24, 4104), (264, 2312), (2056, 136)])
def test_large_bias_of_an_fp32_sum(T, K, N):
    # the bias is added once, to the whole sum. Roundings of the sum: its K values in
    # any order, the six terms of a product, 2 x 2^-22 = 8 U32 for the two left out
    X, W, b, _ = make(T, K, N, hq.F32, seed=9)
    b = 1000.0 * b
    x, w = X.double(), W.double()
    v = x @ w.t().contiguous() + b.double()
    tol = (K + 6 + 8) * U32 * (x.abs() @ w.abs().t().contiguous()) + U32 * v.abs()
    Y = hq.linear(hq.LinearDesc(K, N), X, W, b)
    assert_within(Y, v, tol * (1 + U32) + 1e-30, f"T={T} K={K} N={N}")


@pytest.mark.parametrize("dt,T,K,N", [(hq.BF16, 1_100_003, 8, 2048), (hq.F32, 1_100_003, 16, 2048), (hq.BF16, 2_200_001, 1024, 8)])
def test_more_than_32_bits_of_elements(dt, T, K, N):
    # X or Y has more than 2^31 elements; rows at both ends and around the wraps against calls of their own
    X, W, b, g = make(T, K, N, dt)
    gate = torch.randn(3, N, generator=g, device="cuda").to(DT[dt])
    rows = -(-T // 3)
    desc = hq.LinearDesc(K, N, dt, dt, dt)
    Y = hq.linear(desc, X, W, b, epilogue=hq.Epilogue(hq.HQ_ACT_RELU, gate=gate, gate_rows=rows))
    wide = max(K, N)
    for at in (0, 2 ** 31 // wide - 40, 2 ** 30 // wide - 40, 2 ** 29 // wide - 40, T - 80):
        part = slice(at, at + 80)
        x, w = X[part].double(), W.double()
        v = x @ w.t().contiguous() + b.double()
        err = (K + 16) * U32 * (x.abs() @ w.abs().t().contiguous()) + 8 * U32 * (v.abs() + b.abs().double())
        G = gate[torch.arange(at, at + 80, device="cuda") // rows]
        y, tol = epilogue64(v, err, "relu", dt, None, G, 1)
        assert_within(Y[part], y, tol, f"rows from {at}")
