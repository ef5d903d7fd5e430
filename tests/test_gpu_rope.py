"""hq_rope against float64: head counts and widths, layouts, axes, far and fractional
positions, the norm, in-place and strided rows, the inverse as transpose and inverse,
non-finite rows, neighbours, streams and graph replays.

Tolerance. The angle in [-pi/4, pi/4] is off by 2^-26 pi/2 (the remainder's rounding),
2^-25 (its product) and 2^-25 (the constant): 9e-8, and by 3 x 2^-53 |t| 2 pi / 2 pi in
fp64; the two series by 2^-23 more: 2.2e-7 + |t| 2^-51 on cos and sin. Then a product
pair, 3 U32 (|a| + |b|), behind a norm of 8 squares in a lane, 5 steps across lanes, the
root, the quotient and two products: 12 U32 of each."""
import math

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT, U32, assert_within

pytestmark = pytest.mark.gpu


def rope64(desc, X, positions, freqs, gq=None, gk=None):
    """(y, tolerance before the output's rounding), [T, width] float64."""
    T, H, D = X.shape[0], desc.q_heads + desc.k_heads, desc.head_dim
    x = X[:, : H * D].double().reshape(T, H, D)
    rel = 0.0
    if desc.norm:
        one = torch.ones(D, device=X.device)
        g = torch.cat([(one if gq is None else gq).expand(desc.q_heads, D), (one if gk is None else gk).expand(desc.k_heads, D)])
        x = x / torch.sqrt(x.square().mean(2, keepdim=True) + desc.eps) * g.double()
        rel = 12 * U32
    P = sum(desc.pairs)
    col = [a for a, p in enumerate(desc.pairs) for _ in range(p)]
    t = torch.stack([positions[:, a].double() * freqs[i] for i, a in enumerate(col)], 1)[:, None, :]
    t = -t if desc.inverse else t
    i = torch.arange(P, device=X.device)
    ia, ib = (i, i + P) if desc.layout == hq.HQ_ROPE_HALVES else (2 * i, 2 * i + 1)
    a, b = x[..., ia], x[..., ib]
    y, tol = x.clone(), rel * x.abs()
    y[..., ia], y[..., ib] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    e = (a.abs() + b.abs()) * (2.2e-7 + t.abs() * 2.0 ** -51 + 3 * U32 + rel)
    tol[..., ia], tol[..., ib] = e, e
    return y.reshape(T, H * D), tol.reshape(T, H * D)


def within(Y, y, tol, ydt, what):
    half = torch.finfo(DT[ydt]).eps / 2
    assert_within(Y, y, tol * (1 + half) + half * y.abs() + 1e-30, what)


def make(T, desc, far=1000, seed=0, extra=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7 * T + desc.head_dim)
    width = (desc.q_heads + desc.k_heads) * desc.head_dim
    X = torch.randn(T, width + extra, generator=g, device="cuda").to(DT[desc.x_dtype])
    pos = torch.randint(-far, far, (T, len(desc.pairs)), generator=g, device="cuda", dtype=torch.int32)
    if desc.pos_dtype == hq.HQ_POS_F32:
        pos = pos.float() * 0.328125
    gq, gk = (1.0 + 0.2 * torch.randn(desc.head_dim, generator=g, device="cuda") for _ in range(2))
    return X, pos, hq.rope_freqs(desc), (gq, gk) if desc.norm else (None, None)


def run(T, desc, far=1000, extra=0, seed=0):
    X, pos, f, (gq, gk) = make(T, desc, far, seed, extra)
    Y = hq.rope(desc, X, pos, f, gq, gk)
    assert Y.shape == (T, (desc.q_heads + desc.k_heads) * desc.head_dim) and Y.dtype == DT[desc.y_dtype]
    within(Y, *rope64(desc, X, pos, f, gq, gk), desc.y_dtype, f"T={T} {desc}")
    return Y


LAYOUTS = [hq.HQ_ROPE_PAIRS, hq.HQ_ROPE_HALVES]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,pairs", [(8, (4,)), (16, (3, 5)), (24, (4, 4)), (40, (1, 2, 17)), (64, (32,)), (64, (4, 4, 8)), (72, (18, 18)),
                                     (80, (8, 16, 16)), (96, (0, 48, 0)), (128, (16, 24, 24)), (128, (4, 56, 4)), (160, (20, 20, 20, 20)),
                                     (256, (128,)), (256, (2, 3, 7))])
def test_heads_and_axes(D, pairs, norm, layout):
    for dt in (hq.BF16, hq.F32):
        for q, k in ((1, 0), (0, 1), (3, 2), (16, 16), (32, 8)):
            run(37, hq.RopeDesc(q, k, D, pairs, layout, norm, x_dtype=dt, y_dtype=dt))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 2047, 2048, 2049, 4097])
def test_rows(T):
    for layout in LAYOUTS:
        run(T, hq.RopeDesc(7, 2, 72, (18, 18), layout, True, x_dtype=hq.BF16, y_dtype=hq.BF16))
        run(T, hq.RopeDesc(16, 16, 128, (16, 24, 24), layout, x_dtype=hq.BF16, y_dtype=hq.BF16))


@pytest.mark.parametrize("xdt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("ydt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("pos", [hq.HQ_POS_I32, hq.HQ_POS_F32])
def test_types(xdt, ydt, pos):
    for norm in (False, True):
        for inverse in (False, True):
            if not (norm and inverse):
                run(150, hq.RopeDesc(5, 3, 64, (8, 24), hq.HQ_ROPE_HALVES, norm, inverse=inverse, pos_dtype=pos, x_dtype=xdt, y_dtype=ydt))


@pytest.mark.parametrize("far", [1, 64, 1 << 12, 1 << 20, 1 << 24, 2 ** 31 - 1])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_far_positions(far, layout):
    run(500, hq.RopeDesc(2, 1, 128, (64,), layout), far=far)
    run(500, hq.RopeDesc(2, 1, 128, (64,), layout, pos_dtype=hq.HQ_POS_F32), far=far)


def test_whole_quarters_of_a_turn():
    # angles on and next to the borders of the eighths: frequencies of pi/4 and its neighbours
    d = hq.RopeDesc(1, 0, 16, (8,))
    f = torch.tensor([math.pi / 4, math.pi / 2, math.pi, 2 * math.pi, math.nextafter(math.pi / 4, 1), math.nextafter(math.pi / 4, 0),
                      3 * math.pi / 4, 0.0], dtype=torch.float64, device="cuda")
    pos = torch.arange(-40, 41, device="cuda", dtype=torch.int32)[:, None]
    X = torch.randn(81, 16, device="cuda")
    within(hq.rope(d, X, pos, f), *rope64(d, X, pos, f), hq.F32, "quarters")


def test_position_zero_changes_nothing():
    for dt in (hq.BF16, hq.F32):
        d = hq.RopeDesc(3, 3, 72, (18, 18), x_dtype=dt, y_dtype=dt)
        X, _, f, _ = make(50, d)
        assert torch.equal(hq.rope(d, X, torch.zeros(50, 2, dtype=torch.int32, device="cuda"), f), X)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_inverse_is_the_transpose_and_the_inverse(layout):
    d = hq.RopeDesc(4, 2, 64, (10, 18), layout)
    inv = hq.RopeDesc(4, 2, 64, (10, 18), layout, inverse=True)
    X, pos, f, _ = make(200, d)
    G = make(200, d, seed=5)[0]
    Y, Z = hq.rope(d, X, pos, f), hq.rope(inv, G, pos, f)
    # <R x, g> = <x, R^T g>, row by row: the gradient of the rotation
    a, b = (Y.double() * G.double()).sum(1), (X.double() * Z.double()).sum(1)
    size = (X.double().abs().norm(dim=1) * G.double().norm(dim=1))
    assert ((a - b).abs() <= 4 * (2.2e-7 + 1000 * 2.0 ** -51 + 4 * U32) * size).all()
    back = hq.rope(inv, Y, pos, f)
    per_head = lambda v: v.expand(200, 6, 64).reshape(200, 384)
    pair = per_head(X.double().abs().reshape(200, 6, 64).amax(2, keepdim=True))
    assert ((back.double() - X.double()).abs() <= 8 * (2.2e-7 + 1000 * 2.0 ** -51 + 4 * U32) * pair).all()
    # differences: the map is linear, so (R (x + e g) - R x) / e is R g for any e
    e = 0.5
    diff = (hq.rope(d, X + e * G, pos, f).double() - Y.double()) / e
    direct, tol = rope64(d, G, pos, f)
    both = X.abs() + G.abs()
    big = rope64(d, both, pos, f)[1] + U32 * per_head(both.double().reshape(200, 6, 64).sum(2, keepdim=True))
    assert ((diff - direct).abs() <= 4 * big / e + tol).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_in_place_in_a_packed_projection(dt, norm, layout):
    # q and k turned in place inside [q k v], v and what lies around the rows left alone
    d = hq.RopeDesc(5, 2, 72, (18, 18), layout, norm, x_dtype=dt, y_dtype=dt)
    X, pos, f, (gq, gk) = make(99, d, extra=2 * 72 + 8)
    ref = hq.rope(d, X, pos, f, gq, gk)
    Z = X.clone()
    assert hq.rope(d, Z, pos, f, gq, gk, out=Z) is Z
    assert torch.equal(Z[:, : 7 * 72], ref) and torch.equal(Z[:, 7 * 72:], X[:, 7 * 72:])
    # rows of a wider buffer on both sides
    buf = torch.full((99, 1000), 3.0, device="cuda").to(DT[dt])
    out = buf[:, 8:8 + 7 * 72]
    hq.rope(d, X, pos, f, gq, gk, out=out)
    assert torch.equal(out, ref) and (buf[:, :8] == 3.0).all() and (buf[:, 8 + 7 * 72:] == 3.0).all()


@pytest.mark.parametrize("T", [1, 2])
def test_in_place_by_a_view_of_the_heads(T):
    # X: the q and k columns of a packed row, out: the whole row
    d = hq.RopeDesc(3, 1, 64, (16,), norm=True)
    Z, pos, f, (gq, gk) = make(T, d, extra=64)
    ref = hq.rope(d, Z, pos, f, gq, gk)
    v = Z[:, 256:].clone()
    hq.rope(d, Z[:, :256], pos, f, gq, gk, out=Z)
    assert torch.equal(Z[:, :256], ref) and torch.equal(Z[:, 256:], v)


@pytest.mark.parametrize("D,pairs", [(64, (16, 16)), (72, (20,))])
def test_smallest_eps(D, pairs):
    # heads whose squares are about eps, above it and below the smallest floats
    d = hq.RopeDesc(2, 1, D, pairs, norm=True, eps=2.0 ** -100)
    X, pos, f, (gq, gk) = make(90, d)
    X = (X.view(90, 3, D) * torch.tensor([2.0 ** -50, 2.0 ** -40, 2.0 ** -75], device="cuda")[:, None]).view(90, 3 * D)
    within(hq.rope(d, X, pos, f, gq, gk), *rope64(d, X, pos, f, gq, gk), hq.F32, f"D={D}")


@pytest.mark.parametrize("D,pairs", [(64, (16, 16)), (72, (20,)), (256, (64, 64))])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_squares_past_the_largest_float(D, pairs, dt):
    # beside heads of ordinary size
    d = hq.RopeDesc(5, 3, D, pairs, norm=True, x_dtype=dt, y_dtype=hq.F32)
    X, pos, f, (gq, gk) = make(90, d)
    v = X.view(90, 8, D)
    v[:, 1], v[::2, 6] = v[:, 1] * 2.0 ** 80, v[::2, 6] * 2.0 ** 66
    v[5:9, 4] = torch.where(v[5:9, 4] < 0, -3e38, 3e38)
    within(hq.rope(d, X, pos, f, gq, gk), *rope64(d, X, pos, f, gq, gk), hq.F32, f"D={D} dt={dt}")


def test_non_finite_values_stay_in_their_head():
    d = hq.RopeDesc(4, 2, 64, (16, 16), norm=True)
    X, pos, f, (gq, gk) = make(70, d)
    ref = hq.rope(d, X, pos, f, gq, gk).view(70, 6, 64)
    Z = X.clone().view(70, 6, 64)
    Z[3, 1, 5], Z[40, 5, 0] = float("nan"), float("inf")
    got = hq.rope(d, Z.view(70, -1), pos, f, gq, gk).view(70, 6, 64)
    keep = torch.ones(70, 6, dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[40, 5] = False
    assert torch.equal(got[keep], ref[keep]) and torch.isnan(got[3, 1]).all()
    # a position that is not finite: its row alone, its rotated channels alone
    d = hq.RopeDesc(4, 2, 64, (8, 8), pos_dtype=hq.HQ_POS_F32)
    X, pos, f, _ = make(70, d)
    ref = hq.rope(d, X, pos, f)
    pos[9, 1] = float("inf")
    pos[11, 0] = float("nan")
    got = hq.rope(d, X, pos, f)
    rows = [r for r in range(70) if r not in (9, 11)]
    assert torch.equal(got[rows], ref[rows])
    g9, g11 = got[9].view(6, 64), got[11].view(6, 64)
    assert torch.isnan(g9[:, 16:32]).all() and torch.equal(g9[:, :16], ref[9].view(6, 64)[:, :16])
    assert torch.isnan(g11[:, :16]).all() and torch.equal(g11[:, 16:], ref[11].view(6, 64)[:, 16:])
    assert torch.equal(g9[:, 32:], X[9].view(6, 64)[:, 32:])


def test_offsets_past_32_bits():
    T, d = 300_001, hq.RopeDesc(32, 32, 128, (64,), x_dtype=hq.BF16, y_dtype=hq.BF16)   # 2.5e9 values
    X = torch.zeros(T, 8192, dtype=torch.bfloat16, device="cuda")
    Xe, pe, f, _ = make(64, d)
    X[-64:] = Xe
    pos = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    pos[-64:] = pe
    hq.rope(d, X, pos, f, out=X)
    within(X[-64:], *rope64(d, Xe, pe, f), hq.BF16, "last rows")
    assert (X[:1000] == 0).all()


@pytest.mark.parametrize("T", [3, 700, 5000])
def test_streams_and_graph_replays(T):
    d = hq.RopeDesc(16, 4, 128, (16, 24, 24), hq.HQ_ROPE_HALVES, True, x_dtype=hq.BF16, y_dtype=hq.BF16)
    Xa, pos, f, (gq, gk) = make(T, d)
    Xb = make(T, d, seed=3)[0]
    ref = [hq.rope(d, x, pos, f, gq, gk) for x in (Xa, Xb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, x in enumerate((Xa, Xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.rope(d, x, pos, f, gq, gk))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[k]) for k in range(2) for y in got[k])
    Xg, out = Xa.clone(), torch.empty_like(ref[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hq.rope(d, Xg, pos, f, gq, gk, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.rope(d, Xg, pos, f, gq, gk, out=out)
    for rep in range(4):
        Xg.copy_(Xa if rep % 2 == 0 else Xb)
        graph.replay()
        other = hq.rope(d, Xb, pos, f, gq, gk)
        torch.cuda.synchronize()
        assert torch.equal(out, ref[rep % 2]) and torch.equal(other, ref[1]), f"replay {rep}"
    del graph


def test_empty_and_refusals():
    d = hq.RopeDesc(2, 1, 64, (32,))
    f = hq.rope_freqs(d)
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
    assert hq.rope(d, z(0, 192), z(0, 1, dtype=torch.int32), f).shape == (0, 192)
    X, pos = z(5, 192), z(5, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="positions"):
        hq.rope(d, X, z(5, 1), f)
    with pytest.raises(ValueError, match="positions"):
        hq.rope(d, X, z(4, 1, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="freqs"):
        hq.rope(d, X, pos, f[:16])
    with pytest.raises(ValueError, match="freqs"):
        hq.rope(d, X, pos, f.float())
    with pytest.raises(ValueError, match="shape"):
        hq.rope(d, z(5, 184), pos, f)
    with pytest.raises(ValueError, match="contiguous"):
        hq.rope(d, z(192, 5).t(), pos, f)
    with pytest.raises(hq.HqError, match="without norm"):
        hq.rope(d, X, pos, f, z(64))
    buf = z(7, 192)
    with pytest.raises(hq.HqError, match="overlaps"):
        hq.rope(d, buf[:5], pos, f, out=buf[1:6])
