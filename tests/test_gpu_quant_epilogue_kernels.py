"""hq_quant_linear_epi on every GEMM that it chooses: 32 x 32 outputs per block for few
tokens, 128 x 64 tiles where 128 x 128 would leave CUs idle, 128 x 128 tiles; with the
low-rank branch, both centring modes and fp32 outputs in each; two streams at once and
graph replays. Tolerances as in test_gpu_quant_epilogue."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from test_gpu_quant_epilogue import FORMS, check, epi_of, layer

pytestmark = pytest.mark.gpu

# up to 1024 blocks of 32 x 32 (384 with int8 codes); 9 x 10 tiles of 128 x 128, fewer than CUs; 35 x 10 of them
SIZES = {"few": (300, 1160), "narrow": (1100, 1160), "square": (4353, 1160)}


def build(form, T, N, seed=0):
    kw = dict(FORMS[form])
    return layer(T, kw.pop("K"), N, seed=seed, **kw)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("size", ["narrow", "square"])
def test_values(size, form):
    T, N = SIZES[size]
    desc, prep, X, g = build(form, T, N)
    check(desc, prep, X, "gelu", False, 0, g)
    check(desc, prep, X, "silu", True, -(-T // 3), g, inplace=True)


@pytest.mark.parametrize("form", [f for f in FORMS if not f.startswith("group")])
def test_square_tiles_give_the_plain_calls_bits(form):
    T, N = SIZES["square"]
    desc, prep, X, g = build(form, T, N)
    Y = hq.quant_linear(desc, prep, X)
    assert torch.equal(hq.quant_linear(desc, prep, X, epilogue=hq.Epilogue(residual=torch.zeros_like(Y))), Y)


@pytest.mark.parametrize("form", ["f6_persist_lr1", "f6_channel", "group_bf16", "i8_lr2"])
@pytest.mark.parametrize("size", list(SIZES))
def test_two_streams_at_once(size, form):
    T, N = SIZES[size]
    desc, prep, Xa, g = build(form, T, N)
    Xb = torch.randn(Xa.shape, generator=g, device="cuda").to(Xa.dtype)
    epi = epi_of(T, N, desc.y_dtype, "gelu_tanh", True, 100, g)
    ref = [hq.quant_linear(desc, prep, x, epilogue=epi) for x in (Xa, Xb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for rep in range(4):
        for k, x in enumerate((Xa, Xb)):
            with torch.cuda.stream(streams[k]):
                got[k].append(hq.quant_linear(desc, prep, x, epilogue=epi))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[k]) for k in range(2) for y in got[k])


@pytest.mark.parametrize("form", ["f6_persist_lr1", "f6_channel", "group_bf16", "i8_lr2"])
@pytest.mark.parametrize("size", list(SIZES))
def test_graph_replays(size, form):
    T, N = SIZES[size]
    desc, prep, Xa, g = build(form, T, N)
    Xb = torch.randn(Xa.shape, generator=g, device="cuda").to(Xa.dtype)
    epi = epi_of(T, N, desc.y_dtype, "gelu", True, 300, g)
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
