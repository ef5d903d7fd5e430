"""hq_adapters with operands whose products and sums are whole numbers below 2^24: every
order of every sum is exact, so a piece of A, B or x that a lane reads before another lane
has stored it, or after the next one has taken its place, shows as a wrong number. Ranks
and widths that take one pass through a wave's part of the LDS and several, row by row
and in tiles; rotary positions of more tokens than waves, which reuse their angles' place."""
import pytest
import torch

import hadamard_rotated_bit_amd as hq
from epilogue_ref import DT

pytestmark = pytest.mark.gpu


def whole(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")


def check(T, K, N, r, count, dt, mixed):
    # |u| <= 2 K, |B u| <= 4 K r: below 2^24 for all sizes here; u fits three bf16 parts
    assert 4 * K * r < 2 ** 24
    g = torch.Generator(device="cuda")
    g.manual_seed(T + 7 * K + 13 * N + 17 * r)
    X, A, B = whole(g, -1, 1, T, K), whole(g, -2, 2, count, r, K), whole(g, -2, 2, count, N, r)
    ids = whole(g, -1, count - 1, T)
    if not mixed:
        ids = ids.sort().values
    base = whole(g, -100, 100, T, N)
    want = base.double()
    for a in range(count):
        rows = (ids == a).nonzero().squeeze(1)
        if rows.numel():
            want[rows] += X[rows].double() @ A[a].double().t().contiguous() @ B[a].double().t().contiguous()
    desc = hq.AdapterDesc(K, N, r, dt, dt, hq.F32)
    X, A, B = (t.to(DT[dt]) for t in (X, A, B))
    for _ in range(3):
        Y = hq.adapters(desc, X, A, B, ids.int(), None, base.float())
        wrong = Y.double() != want
        assert not wrong.any(), f"{int(wrong.sum())} wrong, the first at {wrong.nonzero()[0].tolist()}"
    return hq.adapters_workspace_bytes(desc, T) > 0


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 96, 128])
@pytest.mark.parametrize("T,N", [(3, 4360), (24, 1000), (200, 520)])
def test_row_by_row(T, N, r, dt):
    for K in (72, 1032):
        assert not check(T, K, N, r, 5, dt, mixed=True)


@pytest.mark.parametrize("dt", [hq.BF16, hq.F32])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 96, 128])
@pytest.mark.parametrize("T,K", [(2100, 4104), (2080, 136), (9001, 1096)])
def test_tiles(T, K, r, dt):
    for mixed in (False, True):
        assert check(T, K, 392, r, 3, dt, mixed)


@pytest.mark.parametrize("heads,dim,pairs", [(3, 64, (8, 8)), (16, 72, (18, 18)), (2, 256, (64, 64))])
@pytest.mark.parametrize("layout", [hq.HQ_ROPE_PAIRS, hq.HQ_ROPE_HALVES])
def test_rope_of_many_tokens_a_wave(layout, heads, dim, pairs):
    # quarter turns by whole positions: the channels change places and signs, nothing is rounded.
    # 4.2 million tokens and 33 more: the grid's waves take a second token, some of them
    T, P = (1 << 22) + 33, sum(pairs)
    if T * heads * dim > 2 ** 31:
        T = 70001
    desc = hq.RopeDesc(heads, 0, dim, pairs, layout, x_dtype=hq.BF16, y_dtype=hq.BF16)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    X = whole(g, -9, 9, T, heads * dim).to(torch.bfloat16)
    pos = whole(g, 0, 1000, T, len(pairs)).int()
    freqs = torch.full((P,), torch.pi / 2, dtype=torch.float64, device="cuda")
    Y = hq.rope(desc, X, pos, freqs).view(T, heads, dim)
    axis = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).cuda()
    for at in (0, T // 2, T - 5000):   # angles of up to 1000 quarter turns are off by less than 2^-38 of one
        q = (pos[at:at + 5000, axis] % 4)[:, None, :]
        x = X[at:at + 5000].view(-1, heads, dim).float()
        cut = (slice(0, P), slice(P, 2 * P)) if layout == hq.HQ_ROPE_HALVES else (slice(0, 2 * P, 2), slice(1, 2 * P, 2))
        a, b = x[..., cut[0]], x[..., cut[1]]
        c, s = (q == 0).float() - (q == 2).float(), (q == 1).float() - (q == 3).float()
        y = Y[at:at + 5000].float()
        assert ((y[..., cut[0]] - (a * c - b * s)).abs() < 1e-6).all()
        assert ((y[..., cut[1]] - (b * c + a * s)).abs() < 1e-6).all()
        assert torch.equal(y[..., 2 * P:], x[..., 2 * P:])
