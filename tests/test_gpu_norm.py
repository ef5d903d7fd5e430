"""hq_group_norm against float64: group widths of every kind (one channel to
all, not multiples of 8), one position to many, both forms and their borders,
large means, constant and non-finite groups, in-place calls, neighbours,
streams and graph replays.

Tolerance. A group of n values x = mean + std z: fp32 means carry at most a
few roundings of the mean itself (tree sums: 40 U32 max|mean_c| with the lane's
sums of up to 64 values), so (x - mean) / std is off by 40 U32 |mean| / std; the
squares are sums of positive terms about the mean, relative error 40 U32 after
the tree plus the squared mean error; rstd halves it. Then gamma, beta, phi
(epilogue_ref) and one rounding."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import ACTS, DT, U32, act_error, assert_within, phi64

pytestmark = pytest.mark.gpu


def norm64(X, G, gamma, beta, eps, act, ydt):
    S, P, C = X.shape
    x = X.double().view(S, P, G, C // G)
    m = x.mean((1, 3), keepdim=True)
    d = x - m
    var = d.square().mean((1, 3), keepdim=True)
    rs = 1.0 / torch.sqrt(var + eps)
    z = (d * rs)
    top = x.abs().amax((1, 3), keepdim=True)
    # errors of mean, of var (relative) and of the three fp32 steps after them
    em = 40 * U32 * top
    ez = em * rs + z.abs() * (20 * U32 * var * rs * rs + 0.5 * em * em * rs * rs + 4 * U32) + U32 * top * rs
    z, ez = z.reshape(S, P, C), ez.expand(S, P, G, C // G).reshape(S, P, C)
    ga = torch.ones(C, device=X.device).double() if gamma is None else gamma.double()
    be = torch.zeros(C, device=X.device).double() if beta is None else beta.double()
    v = z * ga + be
    ev = ez * ga.abs() + 2 * U32 * (v.abs() + be.abs())
    y = phi64(v, act)
    half = torch.finfo(DT[ydt]).eps / 2
    tol = 1.13 * ev + act_error(v, act, ydt == hq.BF16)
    return y, tol * (1 + half) + half * y.abs() + 1e-30


def make(S, P, C, dt, seed=0, mean=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + S + 31 * P + 17 * C)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    X = (r(S, P, C) * torch.exp(0.5 * r(C)) + mean * r(C)).to(DT[dt])
    return X, 1.0 + 0.2 * r(C), 0.3 * r(C)


def run(S, P, C, G, dt, ydt=None, act="silu", affine=True, inplace=False, mean=1.0, eps=1e-5):
    ydt = dt if ydt is None else ydt
    X, ga, be = make(S, P, C, dt, mean=mean)
    if not affine:
        ga = be = None
    y, tol = norm64(X, G, ga, be, eps, act, ydt)
    desc = hq.NormDesc(C, G, eps, ACTS[act], dt, ydt)
    Y = hq.group_norm(desc, X, ga, be, out=X if inplace else None)
    assert_within(Y.view(-1, C), y.view(-1, C), tol.view(-1, C), f"S={S} P={P} C={C} G={G} dt={dt} ydt={ydt} {act}")
    return Y


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C,G", [(8, 1), (8, 8), (8, 2), (16, 16), (24, 3), (24, 8), (64, 32), (320, 32), (128, 32), (1152, 1),
                                 (1152, 1152), (640, 4), (88, 11), (4096, 1), (4096, 4096), (4096, 32), (2056, 8)])
@pytest.mark.parametrize("S,P", [(1, 1), (3, 2), (2, 77), (1, 1025)])
def test_groups_and_positions(S, P, C, G, dt):
    run(S, P, C, G, dt)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("S,P,C,G", [(8, 1536, 256, 32), (1, 65537, 64, 8), (2, 20011, 320, 32), (5, 4099, 1024, 32),
                                     (700, 130, 64, 4), (9000, 1, 1152, 1), (5000, 3, 40, 8), (1, 9001, 4096, 4096),
                                     (1, 300000, 8, 1)])
def test_sizes(S, P, C, G, dt):
    run(S, P, C, G, dt)


@pytest.mark.parametrize("P", [63, 64, 65, 255, 256, 257, 511, 513, 1023, 1024, 1025, 2047, 2048, 2049, 4097, 8192, 8193])
def test_borders_of_the_forms(P):
    for C, G in ((64, 8), (64, 1), (200, 25)):
        run(2, P, C, G, hq.BF16, act="none")


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("ydt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("act", list(ACTS))
def test_types_activations_affine(act, ydt, dt):
    for S, P in ((2, 40), (1, 6000)):
        run(S, P, 96, 4, dt, ydt, act)
        run(S, P, 96, 4, dt, ydt, act, affine=False)
        if dt == ydt:
            run(S, P, 96, 4, dt, ydt, act, inplace=True)


@pytest.mark.parametrize("S,P", [(2, 40), (1, 6000)])
def test_large_means(S, P):
    # means 1000 times the spread: differences of squares would lose everything
    run(S, P, 64, 8, hq.F32, act="none", mean=1000.0)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("S,P", [(2, 40), (1, 6000)])
def test_constant_group_gives_beta(S, P, dt):
    X = torch.full((S, P, 64), 3.5, device="cuda").to(DT[dt])
    beta = torch.linspace(-1, 1, 64, device="cuda")
    Y = hq.group_norm(hq.NormDesc(64, 8, x_dtype=dt, y_dtype=dt), X, None, beta)
    assert torch.equal(Y, beta.to(DT[dt]).expand(S, P, 64))
    Z = hq.group_norm(hq.NormDesc(64, 8, eps=1.0, x_dtype=dt, y_dtype=dt), torch.zeros_like(X))
    assert bool((Z == 0).all())


@pytest.mark.parametrize("P", [40, 6000])
def test_non_finite_stays_in_its_group(P):
    X, ga, be = make(3, P, 64, hq.BF16)
    desc = hq.NormDesc(64, 8, act=hq.HQ_ACT_SILU, x_dtype=hq.BF16, y_dtype=hq.BF16)
    clean = hq.group_norm(desc, X, ga, be)
    X[1, 7, 9], X[2, 0, 63] = float("nan"), float("inf")
    Y = hq.group_norm(desc, X, ga, be)
    assert bool(torch.isnan(Y[1, :, 8:16]).all()) and bool(torch.isnan(Y[2, :, 56:]).all())
    mask = torch.ones_like(Y, dtype=torch.bool)
    mask[1, :, 8:16] = False
    mask[2, :, 56:] = False
    assert torch.equal(Y[mask], clean[mask])


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("S,P,C,G", [(2, 77, 40, 4), (1, 6001, 72, 9), (3, 1, 8, 1)])
def test_neighbours_are_left_alone(S, P, C, G, dt):
    X, ga, be = make(S, P, C, dt)
    n, pad = X.numel(), 4096
    bx = torch.full((n + 2 * pad,), float("nan"), dtype=DT[dt], device="cuda")
    by = torch.full((n + 2 * pad,), 77.0, dtype=DT[dt], device="cuda")
    x, y = (b[pad:pad + n].view(S, P, C) for b in (bx, by))
    x.copy_(X)
    desc = hq.NormDesc(C, G, x_dtype=dt, y_dtype=dt)
    hq.group_norm(desc, x, ga, be, out=y)
    assert torch.equal(y, hq.group_norm(desc, X, ga, be))
    assert bool((by[:pad] == 77.0).all()) and bool((by[pad + n:] == 77.0).all())


def test_offsets_past_32_bits():
    S, P, C, G = 3, 700_000, 1024, 32    # 2.15e9 values
    X = torch.empty(S, P, C, dtype=torch.bfloat16, device="cuda")
    small, ga, be = make(1, 70_000, C, hq.BF16)
    for s in range(S):
        X[s].view(10, 70_000, C).copy_(small.expand(10, -1, -1))
        X[s] *= s + 1
    desc = hq.NormDesc(C, G, x_dtype=hq.BF16, y_dtype=hq.BF16)
    Y = hq.group_norm(desc, X, ga, be)
    ref, tol = norm64(X[2, -70_000:][None], G, ga, be, 1e-5, "none", hq.BF16)
    assert_within(Y[2, -70_000:], ref[0], tol[0], "last rows of the last sample")


@pytest.mark.parametrize("S,P,C,G", [(2, 77, 320, 32), (1, 20000, 128, 32)])
def test_streams_and_graph_replays(S, P, C, G):
    desc = hq.NormDesc(C, G, act=hq.HQ_ACT_SILU, x_dtype=hq.BF16, y_dtype=hq.BF16)
    Xa, ga, be = make(S, P, C, hq.BF16)
    Xb = make(S, P, C, hq.BF16, seed=5)[0]
    Ya, Yb = hq.group_norm(desc, Xa, ga, be), hq.group_norm(desc, Xb, ga, be)
    n = hq.group_norm_workspace_bytes(desc, S, P)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    Xg, out = Xa.clone(), torch.empty_like(Xa)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hq.group_norm(desc, Xg, ga, be, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, Ya)
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


@pytest.mark.parametrize("S,P,C,G", [(3, 77, 320, 32), (1, 20000, 128, 32), (8, 300, 256, 32)])
def test_two_calls_at_once(S, P, C, G):
    # two streams, each with its own buffers, queued together
    desc = hq.NormDesc(C, G, act=hq.HQ_ACT_SILU, x_dtype=hq.BF16, y_dtype=hq.BF16)
    Xa, ga, be = make(S, P, C, hq.BF16)
    Xb = make(S, P, C, hq.BF16, seed=5)[0]
    ref = [hq.group_norm(desc, x, ga, be) for x in (Xa, Xb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for rep in range(6):
        for k, x in enumerate((Xa, Xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.group_norm(desc, x, ga, be))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[k]) for k in range(2) for y in got[k])


@pytest.mark.parametrize("S,P,C,G,dt", [(1, 1 << 22, 8, 2, hq.BF16), (2, 1 << 20, 40, 4, hq.F32)])
def test_long_sums(S, P, C, G, dt):
    run(S, P, C, G, dt, act="none", mean=3.0)


ROWS = [(8, 1), (24, 1), (24, 3), (64, 8), (64, 4), (512, 1), (520, 1), (1032, 1), (1152, 1), (1152, 18), (1152, 16),
        (1544, 1), (2048, 1), (2056, 1), (2064, 2), (4096, 1), (4096, 2), (4096, 512), (320, 32)]


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C,G", ROWS)
def test_one_position(C, G, dt):
    # layer norm and per-head norms: parts of a wave, whole waves, several pieces per lane, more rows than one turn
    for S in (1, 3, 65):
        run(S, 1, C, G, dt, ydt=hq.F32 if S == 3 else None)
    run(9001 if C <= 1152 else 6001, 1, C, G, dt, inplace=True, mean=30.0)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C,G,value", [(1152, 1, 3.5), (1152, 18, 1000.25), (2056, 1, -0.1)])
def test_constant_rows_give_beta(C, G, value, dt):
    # sums of equal values round, and eps is far below the square of that rounding
    X = torch.full((70, 1, C), value, device="cuda").to(DT[dt])
    beta = torch.linspace(-1, 1, C, device="cuda")
    Y = hq.group_norm(hq.NormDesc(C, G, 1e-12, hq.HQ_ACT_NONE, dt, dt), X, None, beta)
    assert torch.equal(Y, beta.to(DT[dt]).expand(70, 1, C))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_rows_stay_alone(bad):
    # rows that share a wave: a non-finite group is NaN, its neighbours keep their values
    X = torch.randn(40, 1, 64, device="cuda")
    desc = hq.NormDesc(64, 4, 1e-5)
    want = hq.group_norm(desc, X)
    X[7, 0, 20] = bad
    Y = hq.group_norm(desc, X)
    assert torch.isnan(Y[7, 0, 16:32]).all()
    Y[7, 0, 16:32] = want[7, 0, 16:32]
    assert torch.equal(Y, want)


@pytest.mark.parametrize("C,G", [(8, 2), (8, 1)])
def test_more_samples_than_one_grid(C, G):
    # 2^24 blocks of 256 threads are one more thread than a grid holds
    S = (1 << 24) + 5
    X = torch.randn(S, 1, C, device="cuda").to(torch.bfloat16)
    desc = hq.NormDesc(C, G, 1e-5, hq.HQ_ACT_SILU, hq.BF16, hq.BF16)
    Y = hq.group_norm(desc, X)
    for a in (0, (1 << 20) - 50, 1 << 23, S - 100):
        part = X[a:a + 100].contiguous()
        assert torch.equal(Y[a:a + 100], hq.group_norm(desc, part))


@pytest.mark.parametrize("S,P,C,G", [(1_100_003, 1, 2048, 1), (3, 400_000, 2048, 32), (20_000, 60, 2048, 8)])
def test_more_than_32_bits_of_elements(S, P, C, G):
    # samples around the wraps against calls of their own
    X = torch.randn(S, P, C, device="cuda", dtype=torch.bfloat16)
    desc = hq.NormDesc(C, G, 1e-5, hq.HQ_ACT_SILU, hq.BF16, hq.BF16)
    Y = hq.group_norm(desc, X)
    for at in {0, min(S - 1, 2 ** 31 // (P * C)), min(S - 1, 2 ** 30 // (P * C)), S - 1}:
        y, tol = norm64(X[at:at + 1], G, None, None, 1e-5, "silu", hq.BF16)
        assert_within(Y[at].view(-1, C), y.view(-1, C), tol.view(-1, C), f"sample {at}")
