"""hq_rms_norm against float64: widths of every form and their borders, one row to
many, all outputs and types, codes next to and on rounding borders, zero, tiny and
non-finite rows, in-place calls, neighbours, streams and graph replays.

Tolerance. h = x + r is one fp32 rounding. The sum of squares has at most 128
additions in a lane and 9 across lanes and waves (138 U32 of it, halved by the root),
then the mean, the root, the quotient and two products: 75 U32 of y. Codes are equal."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT, U32, assert_within

pytestmark = pytest.mark.gpu

ALL = hq.HQ_RMS_Y | hq.HQ_RMS_SUM | hq.HQ_RMS_CODES


def rms64(x, r, gamma, eps):
    """(h, y, codes, scales) in float64 (codes int8)."""
    h = x.double() if r is None else x.double() + r.double()
    g = torch.ones(x.shape[1], device=x.device).double() if gamma is None else gamma.double()
    rstd = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    v = h * g
    s = v.abs().amax(1, keepdim=True) / 127.0
    codes = torch.where(s > 0, torch.round(v / s), torch.zeros_like(v)).to(torch.int8)
    return h, h * rstd * g, codes, (s * rstd).squeeze(1)


def compare(o, x, r, gamma, eps, ydt, what):
    h, y, codes, scales = rms64(x, r, gamma, eps)
    half = lambda t: torch.finfo(t).eps / 2
    if o.h is not None:
        assert o.h.dtype == x.dtype
        assert_within(o.h, h, (half(x.dtype) + 2 * U32) * h.abs() + 1e-30, what + " h")
    if o.y is not None:
        assert o.y.dtype == DT[ydt]
        assert_within(o.y, y, (75 * U32 * (1 + half(DT[ydt])) + half(DT[ydt])) * y.abs() + 1e-30, what + " y")
    if o.codes is not None:
        assert torch.equal(o.codes, codes), f"{what}: {int((o.codes != codes).sum())} codes differ"
        assert_within(o.scales[:, None], scales[:, None], 80 * U32 * scales[:, None].abs() + 1e-30, what + " scales")


def make(T, C, dt, seed=0, outliers=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7 * T + 13 * C)
    x, r = (torch.randn(T, C, generator=g, device="cuda") for _ in range(2))
    if outliers:
        x[:, torch.randint(0, C, (1 + C // 100,), generator=g, device="cuda")] *= 30.0
    return x.to(DT[dt]), r.to(DT[dt]), 1.0 + 0.2 * torch.randn(C, generator=g, device="cuda")


def run(T, C, dt, outputs=ALL, ydt=None, residual=True, affine=True, eps=1e-6, seed=0):
    ydt = dt if ydt is None else ydt
    x, r, gamma = make(T, C, dt, seed)
    r, gamma = r if residual else None, gamma if affine else None
    o = hq.rms_norm(hq.RmsNormDesc(C, eps, outputs, dt, ydt), x, gamma, r)
    for t, flag in ((o.y, hq.HQ_RMS_Y), (o.h, hq.HQ_RMS_SUM), (o.codes, hq.HQ_RMS_CODES), (o.scales, hq.HQ_RMS_CODES)):
        assert (t is not None) == bool(outputs & flag)
    compare(o, x, r, gamma, eps, ydt, f"T={T} C={C} dt={dt} ydt={ydt} outputs={outputs}")
    return o


WIDTHS = [8, 16, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 1152, 1536, 1544, 2048, 2056, 4096, 4104, 6144, 6152, 8192]


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("C", WIDTHS)
def test_widths_and_rows(C, dt):
    for T in (1, 2, 3, 7, 33, 300):
        run(T, C, dt)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("T,C", [(8192, 1152), (12288, 256), (5001, 72), (20011, 64), (3001, 4096), (70000, 8), (1500, 8192)])
def test_sizes(T, C, dt):
    run(T, C, dt)


@pytest.mark.parametrize("outputs", range(1, 8))
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("ydt", [hq.BF16, hq.F32])
def test_outputs_and_types(outputs, dt, ydt):
    for C in (80, 1160, 4096):
        for residual in (True, False):
            run(50, C, dt, outputs, ydt, residual, affine=residual)
    run(50, 1160, dt, outputs, ydt, True, affine=False, eps=0.5)


@pytest.mark.parametrize("seed", range(8))
def test_codes_are_those_of_exact_arithmetic(seed):
    # 8.4 million codes per seed and type: some 1700 within the fp32 form's reach of a border
    for dt in (hq.BF16, hq.F32):
        run(2048, 4096, dt, hq.HQ_RMS_CODES, seed=100 + seed)
        run(8192, 1024, dt, hq.HQ_RMS_CODES, seed=200 + seed, residual=False)


@pytest.mark.parametrize("C", [64, 256, 512, 1152, 4096])
def test_ties_go_to_the_even_code(C):
    # a maximum of 127 x 2^k gives a scale of 2^k: values (n + 1/2) 2^k are ties, in bf16 and in fp32
    half = torch.arange(-126, 126, device="cuda").float() + 0.5
    row = half.repeat(1 + C // 252)[:C].clone()
    row[C // 2] = -127.0
    x = torch.stack([row * 2.0 ** k for k in (-3, 0, 5, 40, -60, -140, 100)])
    for dt in (hq.F32, hq.BF16):
        v = x.to(DT[dt])
        o = hq.rms_norm(hq.RmsNormDesc(C, 1e-6, ALL, dt, dt), v)
        want = torch.round(v.double() / (v.double().abs().amax(1, keepdim=True) / 127.0)).to(torch.int8)
        assert torch.equal(o.codes, want)
    # a maximum of 3 x 127: a scale of 3, ties at odd multiples of 1.5, reached by a sum of two bf16 values
    # (256 + 125 = 381)
    x = torch.zeros(1, C, device="cuda", dtype=torch.bfloat16)
    r = torch.zeros_like(x)
    x[0, 0], r[0, 0] = 256.0, 125.0
    x[0, 1:60] = 1.5 * (2.0 * torch.arange(1, 60, device="cuda") - 59).to(torch.bfloat16)
    o = hq.rms_norm(hq.RmsNormDesc(C, 1e-6, ALL, hq.BF16, hq.BF16), x, None, r)
    assert torch.equal(o.codes, rms64(x, r, None, 1e-6)[2])


@pytest.mark.parametrize("C", [40, 1152, 4096])
def test_constant_and_zero_rows(C):
    x = torch.tensor([0.0, 3.5, -1e-20, 1e-38, -0.0, 1e-44, 2.0 ** 60], device="cuda")[:, None].expand(7, C).contiguous()
    for dt in (hq.F32, hq.BF16):
        v = x.to(DT[dt])
        o = hq.rms_norm(hq.RmsNormDesc(C, 1e-6, ALL, dt, hq.F32), v)
        assert torch.equal(o.codes, rms64(v, None, None, 1e-6)[2])
        assert torch.isfinite(o.y).all() and torch.isfinite(o.scales).all()
        assert (o.y[0] == 0).all() and o.scales[0] == 0 and (o.y[4] == 0).all()
        assert ((o.y[1] - 1.0).abs() < 1e-6).all() and ((o.y[6] - 1.0).abs() < 1e-6).all()


@pytest.mark.parametrize("C", [40, 1152, 4096])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_smallest_eps(C, dt):
    # rows whose squares are about eps, above it and below the smallest floats
    x, _, gamma = make(60, C, dt)
    x = x * torch.tensor([2.0 ** -50, 2.0 ** -40, 2.0 ** -75], device="cuda").repeat(20)[:, None].to(x.dtype)
    o = hq.rms_norm(hq.RmsNormDesc(C, 2.0 ** -100, ALL, dt, hq.F32), x, gamma)
    compare(o, x, None, gamma, 2.0 ** -100, hq.F32, f"C={C} dt={dt}")


@pytest.mark.parametrize("C", [40, 512, 1152, 4096])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_cancelling_residual(C, dt):
    # h is far smaller than x and r: its rounding is that of the sum, not of its terms
    x, _, gamma = make(60, C, dt)
    r = (-x.float() * (1.0 + 2.0 ** -6)).to(DT[dt])
    o = hq.rms_norm(hq.RmsNormDesc(C, 1e-9, ALL, dt, hq.F32), x, gamma, r)
    compare(o, x, r, gamma, 1e-9, hq.F32, f"C={C} dt={dt}")


@pytest.mark.parametrize("C", [40, 512, 1152, 4096])
def test_non_finite_values_stay_in_their_row(C):
    x, r, gamma = make(9, C, hq.F32)
    desc = hq.RmsNormDesc(C, 1e-6, ALL)
    ref = hq.rms_norm(desc, x, gamma, r)
    bad = x.clone()
    bad[1, C // 2], bad[4, 0], bad[6, C - 1] = float("nan"), float("inf"), -float("inf")
    o = hq.rms_norm(desc, bad, gamma, r)
    ok = [0, 2, 3, 5, 7, 8]
    for a, b in zip(o, ref):
        assert torch.equal(a[ok], b[ok])
    for row in (1, 4, 6):
        assert torch.isnan(o.scales[row]) and (o.codes[row] == 0).all()
    assert torch.isnan(o.y[1]).all()
    assert torch.isnan(o.y[4, 0]) and (o.y[4, 1:] == 0).all() and torch.isnan(o.y[6, C - 1]) and (o.y[6, :-1] == 0).all()
    # a gamma that is not finite
    g2 = gamma.clone()
    g2[3] = float("nan")
    o = hq.rms_norm(desc, x, g2, r)
    assert torch.isnan(o.scales).all() and (o.codes == 0).all()
    assert torch.isnan(o.y[:, 3]).all() and torch.equal(o.y[:, 4:], ref.y[:, 4:])
    # a mean square past the largest float, beside rows of ordinary size
    x[::2] *= 1e25
    compare(hq.rms_norm(desc, x, gamma), x, None, gamma, 1e-6, hq.F32, "large squares")
    x[::2] = torch.where(x[::2] < 0, -3e38, 3e38)
    compare(hq.rms_norm(desc, x, None), x, None, None, 1e-6, hq.F32, "largest squares")


@pytest.mark.parametrize("C", [72, 1152, 4096])
@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
def test_in_place(C, dt):
    desc = hq.RmsNormDesc(C, 1e-6, ALL, dt, dt)
    x, r, gamma = make(40, C, dt)
    ref = hq.rms_norm(desc, x, gamma, r)
    for where in ("residual", "x"):
        a, b = x.clone(), r.clone()
        o = hq.rms_norm(desc, a, gamma, b, sum_out=b if where == "residual" else a, out=a if where == "residual" else b)
        assert o.h.data_ptr() == (b if where == "residual" else a).data_ptr()
        assert all(torch.equal(p, q) for p, q in zip(o, ref))


@pytest.mark.parametrize("C", [8, 72, 1152, 4096, 8192])
def test_memory_around_the_outputs(C):
    T = 5
    x, r, gamma = make(T, C, hq.BF16)
    ref = hq.rms_norm(hq.RmsNormDesc(C, 1e-6, ALL, hq.BF16, hq.BF16), x, gamma, r)
    pad = 64

    def guarded(shape, dtype, fill):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
        return buf, buf[pad:pad + n].view(shape)

    yb, y = guarded((T, C), torch.bfloat16, 7.0)
    hb, h = guarded((T, C), torch.bfloat16, 7.0)
    cb, c = guarded((T, C), torch.int8, 77)
    sb, s = guarded((T,), torch.float32, 7.0)
    o = hq.rms_norm(hq.RmsNormDesc(C, 1e-6, ALL, hq.BF16, hq.BF16), x, gamma, r, out=y, sum_out=h, codes=c, scales=s)
    assert all(torch.equal(p, q) for p, q in zip(o, ref))
    for b, fill in ((yb, 7.0), (hb, 7.0), (cb, 77), (sb, 7.0)):
        assert (b[:pad] == fill).all() and (b[-pad:] == fill).all()


def test_offsets_past_32_bits():
    T, C = 270_001, 8192   # 2.2e9 values
    x = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    xe, _, gamma = make(64, C, hq.BF16)
    x[-64:] = xe
    o = hq.rms_norm(hq.RmsNormDesc(C, 1e-6, hq.HQ_RMS_Y | hq.HQ_RMS_CODES, hq.BF16, hq.BF16), x, gamma)
    tail = hq.RmsNorm(o.y[-64:], None, o.codes[-64:], o.scales[-64:])
    compare(tail, xe, None, gamma, 1e-6, hq.BF16, "last rows")
    assert (o.y[:1000] == 0).all() and (o.codes[:1000] == 0).all() and (o.scales[:1000] == 0).all()


@pytest.mark.parametrize("T,C", [(1, 4096), (300, 1152), (2000, 256)])
def test_streams_and_graph_replays(T, C):
    desc = hq.RmsNormDesc(C, 1e-6, ALL, hq.BF16, hq.BF16)
    xa, r, gamma = make(T, C, hq.BF16)
    xb = make(T, C, hq.BF16, seed=1)[0]
    ref = [hq.rms_norm(desc, x, gamma, r) for x in (xa, xb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, x in enumerate((xa, xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.rms_norm(desc, x, gamma, r))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(p, q) for o in got[k] for p, q in zip(o, ref[k]))
    xg = xa.clone()
    out = [torch.empty_like(t) for t in ref[0]]
    call = lambda: hq.rms_norm(desc, xg, gamma, r, out=out[0], sum_out=out[1], codes=out[2], scales=out[3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        xg.copy_(xa if rep % 2 == 0 else xb)
        graph.replay()
        other = hq.rms_norm(desc, xb, gamma, r)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, ref[rep % 2])), f"replay {rep}"
        assert all(torch.equal(p, q) for p, q in zip(other, ref[1]))
    del graph


def test_empty_and_refusals():
    desc = hq.RmsNormDesc(64, outputs=ALL)
    x = torch.zeros(0, 64, device="cuda")
    o = hq.rms_norm(desc, x)
    assert o.y.shape == (0, 64) and o.codes.shape == (0, 64) and o.scales.shape == (0,)
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="residual"):
        hq.rms_norm(desc, x, residual=torch.zeros(3, 64, device="cuda"))
    with pytest.raises(ValueError, match="gamma"):
        hq.rms_norm(desc, x, torch.zeros(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        hq.rms_norm(desc, torch.zeros(4, 128, device="cuda")[:, :64])
    with pytest.raises(ValueError, match="not among"):
        hq.rms_norm(hq.RmsNormDesc(64), x, codes=torch.zeros(4, 64, device="cuda", dtype=torch.int8))
    with pytest.raises(hq.HqError, match="overlap"):
        hq.rms_norm(desc, x, out=x, sum_out=x)
