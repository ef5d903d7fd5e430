"""hq_quant_linear_epi: the epilogue on every GEMM of the quantised layer (FP6
and int8 engines, group-wise scales, low-rank branch in bf16 and fp32, fp32 and
bf16 outputs, the persistent and the tiled kernels).

The layer's own output V is taken in fp32 from hq_quant_linear of the same
descriptor with y_dtype f32, whose values are exact integers times scales and
the bias terms; the bf16-output kernels form the same V with at most a few
fp32 roundings of terms no larger than |acc s_x s_w| + |b| + |mu c| + |U L2|,
bounded here by 16 U32 of the row's largest |V| plus the largest bias term.
What the epilogue does to V is compared in float64 (epilogue_ref)."""
import dataclasses

import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import ACTS, DT, U32, assert_within, epilogue64

pytestmark = pytest.mark.gpu


def layer(T, K, N, bits, xdt, ydt, center=1, smooth=True, rank=0, gemm=0, group=0, block=64, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + T + K + N)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    desc = hq.Desc(K, N, block, bits, bits, center, smooth, rank, xdt, xdt, ydt, gemm, group)
    X = r(T, K)
    X[:, :3] *= 20.0
    X, W, b = X.to(DT[xdt]), (r(N, K) / K ** 0.5).to(DT[xdt]), 0.1 * r(N)
    sig = hq.sigma(desc, hq.channel_absmax(desc, X), W, 0.5) if smooth else None
    L1 = (0.1 * r(K, rank)).to(DT[xdt]) if rank else None
    L2 = (0.1 * r(rank, N)).to(DT[xdt]) if rank else None
    return desc, hq.prepare(desc, W, b, sig, L1, L2), X, g


def epi_of(T, N, ydt, act, residual, gate_rows, g):
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[ydt])
    R = r(T, N) if residual else None
    G = r(-(-T // gate_rows), 2 * N)[:, N:] if gate_rows else None
    return hq.Epilogue(ACTS[act], R, G, gate_rows)


def check(desc, prep, X, act, residual, gate_rows, g, inplace=False):
    T, N = X.shape[0], desc.d_out
    V = hq.quant_linear(dataclasses.replace(desc, y_dtype=hq.F32), _reheader(desc, prep), X).double()
    views = hq.prepared_views(desc, prep)
    side = views["bias"].abs().max() + (views["c"].abs().max() * 4 if desc.center == 1 else 0)
    err = (16 * U32 * (V.abs().amax(1, keepdim=True) + side.double())).expand(T, N)
    epi = epi_of(T, N, desc.y_dtype, act, residual, gate_rows, g)
    y, tol = epilogue64(V, err, act, desc.y_dtype, epi.residual, epi.gate, gate_rows)
    Y = hq.quant_linear(desc, prep, X, epilogue=epi, out=epi.residual if inplace else None)
    assert_within(Y, y, tol, f"{desc} T={T} {act}")
    return Y


def _reheader(desc, prep):
    # the blob does not depend on y_dtype; only its header names it, and the
    # hot path does not read the header
    return prep


FORMS = {
    "f6_persist": dict(bits=4, xdt=hq.BF16, ydt=hq.BF16, K=1152),
    "f6_persist_lr1": dict(bits=4, xdt=hq.BF16, ydt=hq.BF16, K=640, rank=32),
    "f6_persist_lr2": dict(bits=4, xdt=hq.F32, ydt=hq.BF16, K=640, rank=48),
    "f6_short": dict(bits=4, xdt=hq.BF16, ydt=hq.BF16, K=256, rank=16),
    "f6_f32": dict(bits=4, xdt=hq.F32, ydt=hq.F32, K=640, rank=32),
    "f6_nocenter": dict(bits=4, xdt=hq.BF16, ydt=hq.BF16, K=512, center=0, smooth=False),
    "f6_channel": dict(bits=4, xdt=hq.BF16, ydt=hq.BF16, K=512, center=2),
    "group_bf16": dict(bits=4, xdt=hq.BF16, ydt=hq.BF16, K=384, group=64, rank=32),
    "group_f32": dict(bits=4, xdt=hq.F32, ydt=hq.F32, K=384, group=64),
    "i8": dict(bits=8, xdt=hq.BF16, ydt=hq.BF16, K=1152),
    "i8_lr1": dict(bits=8, xdt=hq.BF16, ydt=hq.BF16, K=640, rank=32),
    "i8_lr2": dict(bits=8, xdt=hq.F32, ydt=hq.BF16, K=640, rank=16),
    "i8_f32": dict(bits=8, xdt=hq.F32, ydt=hq.F32, K=256, center=0, smooth=False),
    "i8_of_4": dict(bits=4, xdt=hq.BF16, ydt=hq.BF16, K=640, gemm=1),
}


@pytest.mark.parametrize("T,N", [(1, 8), (5, 200), (300, 264), (777, 1160)])
@pytest.mark.parametrize("form", list(FORMS))
def test_forms(form, T, N):
    kw = dict(FORMS[form])
    desc, prep, X, g = layer(T, kw.pop("K"), N, **kw)
    print(f"\n[case] {form} T={T} N={N}", flush=True)
    check(desc, prep, X, "gelu", False, 0, g)
    check(desc, prep, X, "none", True, max(1, T // 3), g)
    check(desc, prep, X, "silu", True, 1, g, inplace=True)


@pytest.mark.parametrize("form", ["f6_persist", "f6_persist_lr2", "f6_f32", "i8", "i8_lr2", "group_bf16", "group_f32"])
def test_more_tokens_than_the_few_token_form_takes(form):
    kw = dict(FORMS[form])
    desc, prep, X, g = layer(1201, kw.pop("K"), 1160, **kw)
    check(desc, prep, X, "gelu", True, 400, g)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("K", [128, 1024, 1152, 3584, 8192])
def test_few_tokens(K, bits):
    # fewer stages than waves, one each, one more; several rounds of stages; rows that end inside a tile
    for T, N, rank in ((1, 24, 0), (1, 1152, 64), (31, 40, 16), (33, 264, 0), (100, 136, 48)):
        desc, prep, X, g = layer(T, K, N, bits, hq.BF16, hq.BF16, rank=rank, seed=K)
        check(desc, prep, X, "gelu_tanh", True, 3, g, inplace=True)


@pytest.mark.parametrize("form", list(FORMS))
def test_nothing_to_do_gives_the_plain_calls_bits(form):
    # no epilogue, and a residual of zeros (whatever kernel takes either), at few tokens and at many
    for T, N in ((1, 8), (38, 1160), (300, 264), (1201, 1160)):
        kw = dict(FORMS[form])
        desc, prep, X, g = layer(T, kw.pop("K"), N, **kw)
        Y = hq.quant_linear(desc, prep, X)
        assert torch.equal(hq.quant_linear(desc, prep, X, epilogue=hq.Epilogue()), Y)
        if not desc.group:      # group-wise sums have an order of their own in every kernel
            assert torch.equal(hq.quant_linear(desc, prep, X, epilogue=hq.Epilogue(residual=torch.zeros_like(Y))), Y)


@pytest.mark.parametrize("bits", [4, 8])
def test_few_tokens_are_the_same_rows(bits):
    # a token's outputs do not depend on how many others the call has, whatever kernel takes it
    desc, prep, X, g = layer(3000, 1152, 1160, bits, hq.BF16, hq.BF16)
    epi = hq.Epilogue(hq.HQ_ACT_SILU)
    Y = hq.quant_linear(desc, prep, X, epilogue=epi)
    for T in (1, 40, 700):
        assert torch.equal(hq.quant_linear(desc, prep, X[:T].contiguous(), epilogue=epi), Y[:T])


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("form", ["f6_persist", "f6_f32", "group_bf16", "i8"])
def test_activations(form, act):
    kw = dict(FORMS[form])
    desc, prep, X, g = layer(600, kw.pop("K"), 640, **kw)
    check(desc, prep, X, act, False, 0, g)
    check(desc, prep, X, act, True, 250, g)


@pytest.mark.parametrize("form,T,N", [("f6_persist", 4353, 1160), ("i8", 4353, 1160), ("i8_f32", 2100, 1344), ("i8_f32", 2100, 1160)])
def test_many_tiles(form, T, N):
    kw = dict(FORMS[form])
    desc, prep, X, g = layer(T, kw.pop("K"), N, **kw)
    check(desc, prep, X, "gelu_tanh", True, 1500, g, inplace=True)


@pytest.mark.parametrize("form", ["f6_persist", "group_f32", "i8"])
def test_empty_epilogue_is_the_plain_call(form):
    kw = dict(FORMS[form])
    desc, prep, X, g = layer(700, kw.pop("K"), 520, **kw)
    assert torch.equal(hq.quant_linear(desc, prep, X), hq.quant_linear(desc, prep, X, epilogue=hq.Epilogue()))
    assert hq.quant_linear(desc, prep, X[:0].contiguous(), epilogue=hq.Epilogue(hq.HQ_ACT_SILU)).shape == (0, 520)


@pytest.mark.parametrize("form", ["f6_persist", "f6_f32", "i8"])
def test_neighbours_are_left_alone(form):
    kw = dict(FORMS[form])
    T, N, pad = 301, 520, 4096
    desc, prep, X, g = layer(T, kw.pop("K"), N, **kw)
    epi = epi_of(T, N, desc.y_dtype, "silu", True, 7, g)
    ref = hq.quant_linear(desc, prep, X, epilogue=epi)
    buf = torch.full((T * N + 2 * pad,), 77.0, dtype=DT[desc.y_dtype], device="cuda")
    Y = buf[pad:pad + T * N].view(T, N)
    assert torch.equal(hq.quant_linear(desc, prep, X, out=Y, epilogue=epi), ref)
    assert bool((buf[:pad] == 77.0).all()) and bool((buf[pad + T * N:] == 77.0).all())


def test_graph_replays_match_eager():
    T, N = 900, 1160
    desc, prep, Xa, g = layer(T, 1152, N, 4, hq.BF16, hq.BF16)
    Xb = layer(T, 1152, N, 4, hq.BF16, hq.BF16, seed=9)[2]
    epi = epi_of(T, N, hq.BF16, "gelu", True, 300, g)
    Ya, Yb = (hq.quant_linear(desc, prep, x, epilogue=epi) for x in (Xa, Xb))
    ws = torch.empty(hq.workspace_bytes(desc, T), dtype=torch.uint8, device="cuda")
    Xg, out = Xa.clone(), torch.empty_like(Ya)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hq.quant_linear(desc, prep, Xg, out=out, workspace=ws, epilogue=epi)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.quant_linear(desc, prep, Xg, out=out, workspace=ws, epilogue=epi)
    for rep in range(4):
        Xg.copy_(Xa if rep % 2 == 0 else Xb)
        graph.replay()
        other = hq.quant_linear(desc, prep, Xb, epilogue=epi)
        torch.cuda.synchronize()
        assert torch.equal(out, Ya if rep % 2 == 0 else Yb), f"replay {rep}"
        assert torch.equal(other, Yb)
    del graph


def test_block_of_layers():
    """A denoiser's block half as it is used: group norm with SiLU, the caption
    and modulation layers in 16 bits, the low-bit MLP with GELU, the gated
    low-bit output added into the residual stream in place; against float64 on
    the same low-bit layers' own outputs."""
    S, P, C, H = 2, 320, 512, 1152
    T = S * P
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    bf = torch.bfloat16
    x = r(S, P, C).to(bf)
    nd = hq.NormDesc(C, 32, act=hq.HQ_ACT_SILU, x_dtype=hq.BF16, y_dtype=hq.BF16)
    ga, be = 1 + 0.1 * r(C), 0.1 * r(C)
    emb = r(S, 256).to(bf)
    wt, bt = (r(2 * C, 256) / 16).to(bf), 0.1 * r(2 * C)
    table = hq.linear(hq.LinearDesc(256, 2 * C, hq.BF16, hq.BF16, hq.BF16), emb, wt, bt)
    gate = table[:, C:]
    h = hq.group_norm(nd, x, ga, be).view(T, C)
    w1, w2 = (r(H, C) / C ** 0.5).to(bf), (r(C, H) / H ** 0.5).to(bf)
    d1 = hq.Desc(C, H, 128, 4, 4, 1, False, 0, hq.BF16, hq.BF16, hq.BF16)
    d2 = hq.Desc(H, C, 128, 4, 4, 1, False, 0, hq.BF16, hq.BF16, hq.BF16)
    p1, p2 = hq.prepare(d1, w1, 0.1 * r(H)), hq.prepare(d2, w2, 0.1 * r(C))
    a = hq.quant_linear(d1, p1, h, epilogue=hq.Epilogue(hq.HQ_ACT_GELU_TANH))
    stream = x.view(T, C).clone()
    y = hq.quant_linear(d2, p2, a, epilogue=hq.Epilogue(residual=stream, gate=gate, gate_rows=P), out=stream)
    assert y.data_ptr() == stream.data_ptr()
    # the same steps one by one
    xd = x.double().view(S, P, 32, C // 32)
    z = (xd - xd.mean((1, 3), keepdim=True)) / torch.sqrt(xd.var((1, 3), unbiased=False, keepdim=True) + 1e-5)
    z = z.view(T, C) * ga.double() + be.double()
    href = (z * torch.sigmoid(z))
    assert float((h.double() - href).norm() / href.norm()) < 2 ** -8
    v = hq.quant_linear(d1, p1, h).double()
    aref, tol = epilogue64(v, v.abs() * 2 ** -8, "gelu_tanh", hq.BF16)   # v itself was rounded to bf16
    assert_within(a, aref, tol, "fc1")
    v = hq.quant_linear(d2, p2, a).double()
    tref = emb.double() @ wt.double().t().contiguous() + bt.double()
    assert float((table.double() - tref).norm() / tref.norm()) < 2 ** -8
    yref, tol = epilogue64(v, v.abs() * 2 ** -8, "none", hq.BF16, x.view(T, C), gate, P)
    assert_within(y, yref, tol, "fc2")


@pytest.mark.parametrize("K,T,N", [(128, 1, 8), (256, 33, 40), (384, 64, 1160), (384, 2, 72)])
def test_few_tokens_with_group_scales(K, T, N):
    # at most 6 groups: 6 roundings in the plain call, 1 + 8 here
    for rank in (0, 32):
        desc, prep, X, g = layer(T, K, N, 4, hq.BF16, hq.BF16, rank=rank, group=64, seed=K)
        check(desc, prep, X, "silu", True, 5, g)
