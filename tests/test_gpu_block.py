"""The operators between a block's projections, run together as a block uses them: RMS
norm with the residual into 8-bit codes, an 8-bit qkv layer on the codes, adapters on its
output in place, the norm and rotation of q and k in place. Held to float64 stage by
stage on the stage's own inputs (each stage's tolerance is its own test's), and to the
same bits eagerly, on a side stream and in a replayed graph."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
import test_gpu_adapters as TA
import test_gpu_rms as TR
import test_gpu_rope as TO
from epilogue_ref import epilogue64

pytestmark = pytest.mark.gpu


class Block:
    def __init__(self, T, d, q, k, D, dt=hq.BF16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + T)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        n = (q + 2 * k) * D
        tdt = TA.DT[dt]
        self.norm = hq.RmsNormDesc(d, 1e-6, TR.ALL, dt, dt)
        # rotated stream: the layer takes the codes as they are (block 1, no centring)
        self.layer = hq.Desc(d, n, 1, 8, 8, hq.HQ_CENTER_NONE, False, 0, dt, dt, dt)
        self.lora = hq.AdapterDesc(d, n, 16, dt, dt, dt)
        self.rope = hq.RopeDesc(q, k, D, (D // 4, D // 4), hq.HQ_ROPE_PAIRS, True, x_dtype=dt, y_dtype=dt)
        self.gamma = 1.0 + 0.2 * randn(d)
        self.W, self.b = (randn(n, d) / d ** 0.5).to(tdt), 0.1 * randn(n)
        self.prep = hq.prepare(self.layer, self.W, self.b)
        self.A, self.B = (randn(3, 16, d) / d ** 0.5).to(tdt), (0.25 * randn(3, n, 16)).to(tdt)
        self.ids = (torch.arange(T, device="cuda", dtype=torch.int32) * 4 // max(T, 1)) - 1
        self.scales = 0.5 + torch.rand(3, generator=g, device="cuda")
        self.pos = torch.stack([torch.arange(T, device="cuda") // 16, torch.arange(T, device="cuda") % 16], 1).int()
        self.freqs = hq.rope_freqs(self.rope)
        self.gq, self.gk = (1.0 + 0.2 * randn(D) for _ in range(2))
        self.mu = torch.zeros(T, device="cuda")
        self.x, self.h0 = randn(T, d).to(tdt), randn(T, d).to(tdt)

    def __call__(self, x, h):
        """(qkv, h): h is updated in place, as the residual stream is."""
        o = hq.rms_norm(self.norm, x, self.gamma, h, sum_out=h)
        qkv = hq.gemm_dequant(self.layer, self.prep, o.codes, o.scales, self.mu)
        hq.adapters(self.lora, o.y, self.A, self.B, self.ids, self.scales, qkv, out=qkv)
        hq.rope(self.rope, qkv, self.pos, self.freqs, self.gq, self.gk, out=qkv)
        return qkv, h


@pytest.mark.parametrize("T", [1, 77, 1000])
def test_stage_by_stage(T):
    m = Block(T, 1152, 16, 16, 72)
    h = m.h0.clone()
    o = hq.rms_norm(m.norm, m.x, m.gamma, h, sum_out=h)
    ref = hq.rms_norm(m.norm, m.x, m.gamma, m.h0)
    assert all(torch.equal(a, b) for a, b in zip(o, ref))
    TR.compare(o, m.x, m.h0, m.gamma, 1e-6, hq.BF16, "norm")
    qkv = hq.gemm_dequant(m.layer, m.prep, o.codes, o.scales, m.mu)
    v = hq.prepared_views(m.layer, m.prep)
    wc = v["w_codes"].view(torch.int8).view(-1, 1152).double()
    want = (o.codes.double() @ wc.t().contiguous()) * o.scales.double()[:, None] * v["s_w"].double() + m.b.double()
    # integer sums are exact; three fp32 steps and one rounding to bf16
    tol = 4 * TA.U32 * (want.abs() + m.b.abs().double()) + 2.0 ** -8 * want.abs() + 1e-30
    TA.assert_within(qkv, want, tol, "layer")
    # the codes are the norm to half a step: the layer's output is that of the unquantised one to W8A8's error
    dense = o.y.double() @ m.W.double().t().contiguous() + m.b.double()
    assert (want - dense).norm() < 0.02 * dense.norm()
    base = qkv.clone()
    hq.adapters(m.lora, o.y, m.A, m.B, m.ids, m.scales, qkv, out=qkv)
    y, tol = epilogue64(*TA.adapted64(o.y, m.A, m.B, m.ids, m.scales, base), "none", hq.BF16)
    TA.assert_within(qkv, y, tol, "adapters")
    Z = qkv.clone()
    hq.rope(m.rope, qkv, m.pos, m.freqs, m.gq, m.gk, out=qkv)
    TO.within(qkv[:, : 32 * 72], *TO.rope64(m.rope, Z, m.pos, m.freqs, m.gq, m.gk), hq.BF16, "rope")
    assert torch.equal(qkv[:, 32 * 72:], Z[:, 32 * 72:])
    h2 = m.h0.clone()
    got, h2 = m(m.x, h2)
    assert torch.equal(got, qkv) and torch.equal(h2, h)


@pytest.mark.parametrize("T", [3, 500])
def test_stream_and_graph(T):
    m = Block(T, 1024, 8, 2, 64)
    h = m.h0.clone()
    ref, href = m(m.x, h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = m.h0.clone()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        got, _ = m(m.x, h)
    side.synchronize()
    assert torch.equal(got, ref) and torch.equal(h, href)
    graph = torch.cuda.CUDAGraph()
    hg = m.h0.clone()
    with torch.cuda.graph(graph):
        out, _ = m(m.x, hg)
    for _ in range(4):
        hg.copy_(m.h0)
        graph.replay()
        other, _ = m(m.x, m.h0.clone())
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(hg, href) and torch.equal(other, ref)
    del graph
