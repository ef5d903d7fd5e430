"""hq_adapters against float64: one row to many, ragged widths, every rank, rows of
mixed adapters, of runs and of none, ids outside the range, the epilogue's parts, base
in place or absent, non-finite rows, neighbours, streams and graph replays, row by row
(no workspace) and in tiles of rows (with one).

Tolerance. u = A x sums K products in fp32 in some order: K + 1 roundings of the
absolute products, one more for the scale. B u sums `rank` products: rank + 4 roundings
of the absolute ones (u may be cut into exact parts). base is added once; then
epilogue_ref."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import ACTS, DT, U32, assert_within, epilogue64

pytestmark = pytest.mark.gpu


def adapted64(X, A, B, ids, scales, base):
    """(V, error) in float64, adapter by adapter."""
    T, N, K, r = X.shape[0], B.shape[1], X.shape[1], A.shape[1]
    v = torch.zeros(T, N, device=X.device).double() if base is None else base.double()
    err = torch.zeros_like(v)
    for i in range(A.shape[0]):
        rows = (ids == i).nonzero().squeeze(1)
        if rows.numel() == 0:
            continue
        x, a, b = X[rows].double(), A[i].double().t().contiguous(), B[i].double().t().contiguous()
        s = 1.0 if scales is None else scales[i].double()
        u = x @ a * s
        ue = (K + 2) * U32 * (x.abs() @ a.abs()) * abs(s) + U32 * u.abs()
        v[rows] += u @ b
        err[rows] = ue @ b.abs() + (r + 4) * U32 * (u.abs() @ b.abs())
    return v, err + U32 * v.abs()


def make(T, K, N, r, count, dt, ydt=None, kind="runs", seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + T + 7 * K + 13 * N + r)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    X = randn(T, K).to(DT[dt])
    A, B = (randn(count, r, K) / K ** 0.5).to(DT[dt]), (randn(count, N, r) / r ** 0.5).to(DT[dt])
    base = randn(T, N).to(DT[dt if ydt is None else ydt])
    scales = 0.5 + torch.rand(count, generator=g, device="cuda")
    if kind == "mixed":
        ids = torch.randint(-1, count, (T,), generator=g, device="cuda")
    elif kind == "one":
        ids = torch.zeros(T, device="cuda") + count // 2
    elif kind == "none":
        ids = torch.full((T,), -1, device="cuda")
    else:   # runs of ragged lengths
        cuts = torch.randint(0, T + 1, (max(1, min(T, 2 * count)),), generator=g, device="cuda")
        run_of = (torch.arange(T, device="cuda")[:, None] >= cuts[None, :]).sum(1)
        ids = torch.randint(-1, count, (cuts.numel() + 1,), generator=g, device="cuda")[run_of]
    return X, A, B, ids.int(), scales, base, g


def run(T, K, N, r, count=3, dt=hq.BF16, ydt=None, kind="runs", act="none", residual=False, gate_rows=0, scaled=True,
        based=True, inplace=None, seed=0):
    ydt = dt if ydt is None else ydt
    X, A, B, ids, scales, base, g = make(T, K, N, r, count, dt, ydt, kind, seed)
    scales, base = scales if scaled else None, base if based else None
    R = torch.randn(T, N, generator=g, device="cuda").to(DT[ydt]) if residual else None
    G = torch.randn(-(-T // gate_rows), 2 * N, generator=g, device="cuda").to(DT[ydt])[:, N:] if gate_rows else None
    v, err = adapted64(X, A, B, ids, scales, base)
    y, tol = epilogue64(v, err, act, ydt, R, G, gate_rows)
    out = {"base": base, "residual": R, None: None}[inplace]
    Y = hq.adapters(hq.AdapterDesc(K, N, r, dt, dt, ydt), X, A, B, ids, scales, base,
                    hq.Epilogue(ACTS[act], R, G, gate_rows) if act != "none" or residual or gate_rows else None, out=out)
    assert Y.dtype == DT[ydt] and (out is None or Y is out)
    assert_within(Y, y, tol, f"T={T} K={K} N={N} r={r} n={count} dt={dt} ydt={ydt} {kind} {act}")
    return Y


def in_tiles(T, K, N, r, dt):
    return hq.adapters_workspace_bytes(hq.AdapterDesc(K, N, r, dt, dt, dt), T) > 0


ROWS = [1, 2, 3, 5, 15, 16, 17, 31, 33, 63, 64, 65, 130, 257, 300]


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("K,N", [(8, 8), (16, 24), (72, 136), (256, 1152), (1160, 264)])
@pytest.mark.parametrize("kind", ["runs", "mixed"])
def test_rows_and_widths(kind, K, N, dt):
    for T in ROWS:
        run(T, K, N, 16, dt=dt, kind=kind)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("K,N", [(8, 8), (16, 24), (72, 136), (136, 128), (264, 392)])
@pytest.mark.parametrize("kind", ["runs", "mixed", "one"])
def test_tiles_and_widths(kind, K, N, dt):
    for T in (2049, 2063, 2064, 2065, 2079, 2081, 2111, 2112, 2113, 2300):
        assert in_tiles(T, K, N, 16, dt)
        run(T, K, N, 16, dt=dt, kind=kind)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("r", list(range(8, 129, 8)))
def test_ranks(r, dt):
    for T, kind in ((1, "one"), (24, "mixed"), (200, "runs"), (2049, "runs"), (2100, "mixed")):
        assert in_tiles(T, 328, 456, r, dt) == (T > 2000)
        run(T, 328, 456, r, 4, dt, kind=kind)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,K,N,r", [(65, 4096, 4096, 128), (257, 4096, 2048, 64), (300, 8200, 520, 128), (513, 6152, 3080, 24),
                                     (1100, 2056, 2056, 64)])
def test_few_tiles_share_their_k(T, K, N, r, dt):
    # u in several parts, chunks that end inside a row
    for kind in ("runs", "mixed"):
        run(T, K, N, r, 5, dt, kind=kind)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,K,N,r,n,kind", [(24, 4096, 4096, 16, 16, "mixed"), (1037, 1160, 2312, 8, 5, "runs"),
                                            (4097, 1152, 4608, 32, 4, "runs"), (2500, 4096, 520, 64, 6, "runs"),
                                            (300, 8200, 64, 128, 3, "one"), (9000, 64, 128, 16, 64, "mixed"),
                                            (513, 136, 8200, 24, 2, "one"), (64, 2048, 2048, 16, 64, "mixed")])
def test_sizes(T, K, N, r, n, kind, dt):
    run(T, K, N, r, n, dt, kind=kind)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("ydt", [hq.BF16, hq.F32])
def test_types_and_epilogues(act, dt, ydt):
    for T in (7, 90, 2100):
        run(T, 72, 200, 16, 3, dt, ydt, act=act)
        run(T, 72, 200, 16, 3, dt, ydt, act=act, residual=True, gate_rows=T // 3 + 1)
        run(T, 72, 200, 16, 3, dt, ydt, act=act, residual=True, inplace="residual")
        run(T, 72, 200, 16, 3, dt, ydt, act=act, gate_rows=1, inplace="base")
        run(T, 72, 200, 16, 3, dt, ydt, act=act, scaled=False, based=False)


@pytest.mark.parametrize("T", [3, 200, 2100])
def test_large_base_is_added_once(T):
    # what the adapter adds is summed by itself: a base a thousand times as large rounds it once
    X, A, B, ids, scales, base, _ = make(T, 264, 392, 128, 3, hq.F32)
    base = 1000.0 * base
    y, tol = epilogue64(*adapted64(X, A, B, ids, scales, base), "none", hq.F32)
    assert_within(hq.adapters(hq.AdapterDesc(264, 392, 128), X, A, B, ids, scales, base), y, tol, f"T={T}")


@pytest.mark.parametrize("T", [2, 2100])
def test_parts_of_u_are_exact(T):
    # a bf16 product of u = a few large and a few small parts that cancel in B u: an error of 2^-16 or
    # of 2^-8 of u would be all that is left
    K, N, r = 64, 128, 16
    X = torch.ones(T, K, device="cuda", dtype=torch.bfloat16)
    A = torch.zeros(1, r, K, device="cuda", dtype=torch.bfloat16)
    A[0, 0, 0], A[0, 0, 1], A[0, 0, 2] = 1.0, 2.0 ** -9, 2.0 ** -18
    A[0, 1, 0], A[0, 1, 1] = 1.0, 2.0 ** -9
    B = torch.zeros(1, N, r, device="cuda", dtype=torch.bfloat16)
    B[0, :, 0], B[0, :, 1] = 1.0, -1.0
    Y = hq.adapters(hq.AdapterDesc(K, N, r, hq.BF16, hq.BF16, hq.F32), X, A, B, torch.zeros(T, dtype=torch.int32, device="cuda"))
    assert (Y == 2.0 ** -18).all()


@pytest.mark.parametrize("T", [1, 40, 600, 3000])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_rows_without_an_adapter(T, dt):
    # base passes unchanged, in place or not, and x is not looked at
    X, A, B, ids, scales, base, _ = make(T, 264, 392, 16, 3, dt, kind="none")
    X[:] = float("nan")
    ids = torch.tensor([-1, 3, 2 ** 31 - 1, -2 ** 31, 4], device="cuda", dtype=torch.int32).repeat(T)[:T].contiguous()
    desc = hq.AdapterDesc(264, 392, 16, dt, dt, dt)
    assert torch.equal(hq.adapters(desc, X, A, B, ids, scales, base), base)
    assert (hq.adapters(desc, X, A, B, ids, scales) == 0).all()
    keep = base.clone()
    hq.adapters(desc, X, A, B, ids, scales, base, out=base)
    assert torch.equal(base, keep)
    # no adapter loaded at all
    assert torch.equal(hq.adapters(desc, X, A[:0].contiguous(), B[:0].contiguous(), ids, None, base), base)


@pytest.mark.parametrize("T", [40, 600, 2100])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_non_finite_values_stay_in_their_row_and_adapter(T, dt):
    X, A, B, ids, scales, base, _ = make(T, 264, 392, 16, 4, dt, kind="mixed")
    ids[:] = torch.arange(T, device="cuda", dtype=torch.int32) % 4 - 1   # -1, 0, 1, 2
    desc = hq.AdapterDesc(264, 392, 16, dt, dt, dt)
    ref = hq.adapters(desc, X, A, B, ids, scales, base)
    Z = X.clone()
    Z[5, 3], Z[18, 0], Z[0, 7] = float("nan"), float("inf"), float("nan")   # row 0 has no adapter
    got = hq.adapters(desc, Z, A, B, ids, scales, base)
    rows = [t for t in range(T) if t not in (5, 18)]
    assert torch.equal(got[rows], ref[rows]) and torch.isnan(got[5]).all() and not torch.isfinite(got[18]).any()
    # an adapter that is not finite: its rows alone (one that no row has: none)
    A2, B2 = A.clone(), B.clone()
    A2[1, 2, 5], A2[3], B2[3] = float("nan"), float("nan"), float("inf")
    got = hq.adapters(desc, X, A2, B2, ids, scales, base)
    assert torch.isnan(got[ids == 1]).all() and torch.equal(got[ids != 1], ref[ids != 1])


@pytest.mark.parametrize("T,K,N,r", [(1, 8, 8, 8), (5, 72, 136, 16), (33, 264, 200, 24), (700, 72, 136, 40), (2049, 72, 136, 40),
                                     (2063, 8, 8, 8), (2100, 264, 200, 72), (2049, 136, 264, 128)])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_memory_around_the_operands(T, K, N, r, dt):
    # what lies around X, A and B does not enter, what lies around Y and the workspace stays
    X, A, B, ids, scales, base, _ = make(T, K, N, r, 2, dt)
    desc = hq.AdapterDesc(K, N, r, dt, dt, dt)
    ref = hq.adapters(desc, X, A, B, ids, scales, base)

    def framed(t, fill, pad=64):
        buf = torch.full((t.numel() + 2 * pad,), fill, dtype=t.dtype, device="cuda")
        view = buf[pad:pad + t.numel()].view(t.shape)
        view.copy_(t)
        return buf, view

    (_, Xf), (_, Af), (_, Bf), (_, bf) = (framed(t, float("nan")) for t in (X, A, B, base))
    yb, Y = framed(torch.zeros_like(base), 5.0)
    n = hq.adapters_workspace_bytes(desc, T)
    wb, ws = framed(torch.zeros(n, dtype=torch.uint8, device="cuda"), 99)
    _, idf = framed(ids, 1)
    hq.adapters(desc, Xf, Af, Bf, idf, scales, bf, out=Y, workspace=ws if n else None)
    assert torch.equal(Y, ref)
    assert (yb[:64] == 5.0).all() and (yb[-64:] == 5.0).all() and (wb[:64] == 99).all() and (wb[-64:] == 99).all()


@pytest.mark.parametrize("dt,T,K,N", [(hq.BF16, 270_001, 8192, 8), (hq.BF16, 270_001, 8, 8192)])
def test_offsets_past_32_bits(dt, T, K, N):
    desc = hq.AdapterDesc(K, N, 8, dt, dt, dt)
    X, A, B, _, scales, _, g = make(1, K, N, 8, 3, dt)
    X = torch.randn(T, K, generator=g, device="cuda", dtype=torch.float32 if K == 8 else torch.bfloat16).to(DT[dt])
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) // 1000) % 4 - 1
    Y = hq.adapters(desc, X, A, B, ids, scales)
    for at in (0, 2 ** 31 // 8192 - 40, 2 ** 30 // 8192 - 40, 2 ** 29 // 8192 - 40, T - 80):
        part = slice(at, at + 80)
        assert_within(Y[part], *epilogue64(*adapted64(X[part], A, B, ids[part], scales, None), "none", dt), f"rows from {at}")


@pytest.mark.parametrize("T,K,N,r,kind", [(1, 1152, 4608, 16, "one"), (24, 4096, 1152, 16, "mixed"), (1000, 1160, 2312, 32, "runs"),
                                          (2500, 264, 520, 64, "mixed")])
def test_streams_and_graph_replays(T, K, N, r, kind):
    desc = hq.AdapterDesc(K, N, r, hq.BF16, hq.BF16, hq.BF16)
    Xa, A, B, ids, scales, base, _ = make(T, K, N, r, 4, hq.BF16, kind=kind)
    Xb = make(T, K, N, r, 4, hq.BF16, kind=kind, seed=1)[0]
    epi = hq.Epilogue(hq.HQ_ACT_GELU_TANH)
    ref = [hq.adapters(desc, x, A, B, ids, scales, base, epi) for x in (Xa, Xb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, x in enumerate((Xa, Xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.adapters(desc, x, A, B, ids, scales, base, epi))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[k]) for k in range(2) for y in got[k])
    n = hq.adapters_workspace_bytes(desc, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    Xg, out = Xa.clone(), torch.empty_like(base)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hq.adapters(desc, Xg, A, B, ids, scales, base, epi, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.adapters(desc, Xg, A, B, ids, scales, base, epi, out=out, workspace=ws)
    for rep in range(4):
        Xg.copy_(Xa if rep % 2 == 0 else Xb)
        graph.replay()
        other = hq.adapters(desc, Xb, A, B, ids, scales, base, epi)
        torch.cuda.synchronize()
        assert torch.equal(out, ref[rep % 2]) and torch.equal(other, ref[1]), f"replay {rep}"
    del graph


def test_empty_and_refusals():
    d = hq.AdapterDesc(64, 128, 8)
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
    A, B = z(2, 8, 64), z(2, 128, 8)
    i = lambda n: z(n, dtype=torch.int32)
    assert hq.adapters(d, z(0, 64), A, B, i(0)).shape == (0, 128)
    X = z(5, 64)
    for bad, word in ((dict(A=z(2, 16, 64)), "A must"), (dict(A=z(8, 64)), "A must"), (dict(B=z(3, 128, 8)), "B must"),
                      (dict(ids=i(4)), "ids"), (dict(ids=z(5, dtype=torch.int64)), "ids"), (dict(scales=z(3)), "scales"),
                      (dict(base=z(5, 120)), "base"), (dict(out=z(4, 128)), "out"), (dict(A=A.bfloat16()), "A must")):
        kw = dict(A=A, B=B, ids=i(5))
        kw.update(bad)
        with pytest.raises(ValueError, match=word):
            hq.adapters(d, X, **kw)
    buf = z(6, 128)
    with pytest.raises(hq.HqError, match="Y overlaps"):
        hq.adapters(d, X, A, B, i(5), base=buf[:5], out=buf[1:])
