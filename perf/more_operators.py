"""The operators between the projections of a transformer block, as they are measured.

* ``rms_norm``: h = x + r and the root-mean-square norm of h, in 16 or 32 bits and as the 8-bit codes
  with a scale per row that an 8-bit layer takes.
* ``adapters``: phi(base + s_a B_a (A_a x)), low-rank adapters of many requests beside a projection that
  they share, the adapter a chosen row by row (or none).
* ``rope``: rotary positions with several axes (time, height, width) on the q and k heads of a packed
  projection, behind an RMS norm of each head where the model has one.

Each has a plain form in elementary torch operations (``own`` false) and the framework's call
(``own`` true). Inputs come from the seed alone.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rms(name, T, C, dtype, residual, outputs):
    """outputs: of "h" (the sum), "y" (the norm) and "q" (its codes and scales)."""
    return {"name": name, "op": "rms_norm", "T": T, "C": C, "dtype": dtype, "residual": residual, "outputs": outputs}


def _rope(name, T, q_heads, k_heads, head_dim, pairs, halves, norm, dtype, far, whole, inverse=False):
    """pairs: rotated pairs of each axis; far: positions are below it; whole: positions are integers;
    inverse: by the negative angles (back to no position; the transposed map)."""
    return {"name": name, "op": "rope", "T": T, "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
            "pairs": pairs, "halves": halves, "norm": norm, "dtype": dtype, "far": far, "whole": whole, "inverse": inverse}


def _adapters(name, T, d_in, d_out, rank, count, dtype, act, mixed):
    """count: adapters loaded; mixed: each row has its own adapter (decoding), else rows come in runs."""
    return {"name": name, "op": "adapters", "T": T, "d_in": d_in, "d_out": d_out, "rank": rank, "count": count,
            "dtype": dtype, "act": act, "mixed": mixed}


def listed():
    return [
        # one token on its way into a block: nothing but latency
        _rms("rms_step", 1, 4096, "bf16", True, "hy"),
        # two images of 4096 tokens, the sum kept, the norm only as codes for an 8-bit layer
        _rms("rms_block_codes", 8192, 1152, "bf16", True, "hq"),
        # 8 latents of the image codec in 32 bits, no residual
        _rms("rms_codec_f32", 12288, 256, "f32", False, "yq"),
        # the square projection's input: sum, norm for the 16-bit branch, codes for the 8-bit layer
        _rms("rms_wide", 8192, 4096, "bf16", True, "hyq"),
        # three requests decoding one token each, far into a long sequence
        _rope("rope_step", 3, 32, 8, 128, "16,24,24", True, True, "bf16", 1 << 20, True),
        # two images of 64 x 64 patches, 16 heads of 72 channels, rows and columns
        _rope("rope_image", 8192, 16, 16, 72, "18,18", False, True, "bf16", 64, True),
        # an odd count of tokens in 32 bits, half of each head turned back, positions between the integers
        _rope("rope_ragged_f32", 1037, 5, 3, 64, "8,8", True, False, "f32", 4096, False, inverse=True),
        # a video of 16 frames of 32 x 48 patches at a frame rate that is not the trained one
        _rope("rope_video", 24576, 16, 16, 128, "16,24,24", False, True, "bf16", 512, False),
        # 24 requests decoding one token each through 16 loaded adapters
        _adapters("adapters_step", 24, 4096, 4096, 16, 16, "bf16", "none", True),
        # sizes that fill no tile, in 32 bits
        _adapters("adapters_ragged_f32", 1037, 1160, 2312, 8, 5, "f32", "silu", False),
        # the MLP input layer of a block, images of several requests in one batch
        _adapters("adapters_image", 8192, 1152, 4608, 32, 4, "bf16", "gelu_tanh", False),
        # the square projection under adapters of a large rank
        _adapters("adapters_wide", 8192, 4096, 4096, 64, 6, "bf16", "none", False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step + 0.5) * step)


def draw(rng):
    op = rng.choice(("rms_norm", "rope", "adapters"))
    if op == "rms_norm":
        while True:
            T, C = _log(rng, 1, 16384), _log(rng, 64, 8192, 8)
            if T * C <= 8192 * 4096:
                break
        return {"op": op, "T": T, "C": C, "dtype": rng.choice(("bf16", "bf16", "f32")), "residual": rng.random() < 0.7,
                "outputs": rng.choice(("y", "hy", "q", "hq", "yq", "hyq"))}
    if op == "rope":
        while True:
            T, q, dim = _log(rng, 1, 24576), rng.randint(1, 32), rng.choice((32, 64, 72, 80, 96, 128, 256))
            k = rng.choice((q, max(1, q // 4), 0))
            if T * (q + k) * dim <= 24576 * 4096:
                break
        half = dim // 2 if rng.random() < 0.7 else 4 * rng.randint(1, dim // 8)
        axes = rng.choice((1, 2, 3))
        cuts = sorted(rng.randint(0, half) for _ in range(axes - 1))
        pairs = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        norm = rng.random() < 0.6
        return {"op": op, "T": T, "q_heads": q, "k_heads": k, "head_dim": dim, "pairs": ",".join(map(str, pairs)),
                "halves": rng.random() < 0.5, "norm": norm, "dtype": rng.choice(("bf16", "bf16", "f32")),
                "far": _log(rng, 16, 1 << 22), "whole": rng.random() < 0.6, "inverse": not norm and rng.random() < 0.4}
    while True:
        T, k, n = _log(rng, 1, 8192), _log(rng, 64, 4608, 8), _log(rng, 64, 4608, 8)
        rank, count = rng.choice((8, 16, 16, 24, 32, 64, 128)), _log(rng, 1, 64)
        if T * (k + 2 * n) <= 8192 * 12288 and T * (k + n) * rank * count <= 8192 * 8192 * 384:
            break
    return {"op": op, "T": T, "d_in": k, "d_out": n, "rank": rank, "count": count, "dtype": rng.choice(("bf16", "bf16", "f32")),
            "act": rng.choice(("none", "none", "silu", "gelu_tanh")), "mixed": T <= 256 and rng.random() < 0.6}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pairs(case):
    return [int(p) for p in case["pairs"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st, T, dt = {"case": case}, case["T"], DTYPES[case["dtype"]]
    if case["op"] == "rms_norm":
        C = case["C"]
        x = _randn(g, T, C)
        x[:, torch.randint(0, C, (max(1, C // 100),), generator=g, device="cuda")] *= 30.0  # outlier channels
        st["x"] = x.to(dt)
        st["residual"] = _randn(g, T, C).to(dt) if case["residual"] else None
        st["gamma"] = 1.0 + 0.2 * _randn(g, C)
    elif case["op"] == "rope":
        dim, pairs = case["head_dim"], _pairs(case)
        heads = case["q_heads"] + case["k_heads"]
        # the packed projection: q, k and (as wide as k) v of a token in one row
        st["x"] = _randn(g, T, (heads + case["k_heads"]) * dim).to(dt)
        st["positions"] = torch.randint(0, case["far"], (T, len(pairs)), generator=g, device="cuda", dtype=torch.int32)
        if not case["whole"]:
            st["positions"] = st["positions"].float() * 0.53125
        # theta^(-i / p) for pair i of an axis of p pairs
        st["freqs"] = torch.cat([torch.pow(torch.tensor(10000.0, dtype=torch.float64),
                                           -torch.arange(p, dtype=torch.float64) / p) for p in pairs if p]).cuda()
        norm = case["norm"]
        st["gamma_q"] = 1.0 + 0.2 * _randn(g, dim) if norm else None
        st["gamma_k"] = 1.0 + 0.2 * _randn(g, dim) if norm and case["k_heads"] else None
    else:
        k, n, r, count = case["d_in"], case["d_out"], case["rank"], case["count"]
        st["x"], st["base"] = _randn(g, T, k).to(dt), _randn(g, T, n).to(dt)
        st["a"] = (_randn(g, count, r, k) / math.sqrt(k)).to(dt)
        st["b"] = (_randn(g, count, n, r) / math.sqrt(r)).to(dt)
        st["scales"] = 0.5 + torch.rand(count, generator=g, device="cuda")
        # -1: a request without an adapter
        if case["mixed"]:
            ids = torch.randint(-1, count, (T,), generator=g, device="cuda")
        else:
            cuts = torch.randint(0, T + 1, (min(2 * count, T),), generator=g, device="cuda")
            run_of = (torch.arange(T, device="cuda")[:, None] >= cuts[None, :]).sum(1)
            ids = torch.randint(-1, count, (cuts.numel() + 1,), generator=g, device="cuda")[run_of]
        st["ids"] = ids.int()
    if own:
        st["desc"] = _desc(case)
    return st


def _desc(case):
    """What a program of the framework keeps for the operator: its descriptor (and the adapters' epilogue)."""
    import hadamard_rotated_bit_amd as hq
    dt = {"f32": hq.F32, "bf16": hq.BF16}[case["dtype"]]
    if case["op"] == "rms_norm":
        out = {"h": hq.HQ_RMS_SUM, "y": hq.HQ_RMS_Y, "q": hq.HQ_RMS_CODES}
        return hq.RmsNormDesc(case["C"], eps=1e-6, outputs=sum(out[o] for o in case["outputs"]), x_dtype=dt, y_dtype=dt)
    if case["op"] == "rope":
        return hq.RopeDesc(case["q_heads"], case["k_heads"], case["head_dim"], tuple(_pairs(case)),
                           layout=hq.HQ_ROPE_HALVES if case["halves"] else hq.HQ_ROPE_PAIRS, norm=case["norm"], eps=1e-6,
                           inverse=case["inverse"], pos_dtype=hq.HQ_POS_I32 if case["whole"] else hq.HQ_POS_F32, x_dtype=dt, y_dtype=dt)
    act = {"none": hq.HQ_ACT_NONE, "silu": hq.HQ_ACT_SILU, "gelu_tanh": hq.HQ_ACT_GELU_TANH}[case["act"]]
    return (hq.AdapterDesc(case["d_in"], case["d_out"], case["rank"], x_dtype=dt, w_dtype=dt, y_dtype=dt),
            hq.Epilogue(act=act) if case["act"] != "none" else None)


def run(st):
    case = st["case"]
    if own:
        import hadamard_rotated_bit_amd as hq
        if case["op"] == "rms_norm":
            o = hq.rms_norm(st["desc"], st["x"], st["gamma"], residual=st["residual"])
            return {"h": o.h, "y": o.y, "codes": o.codes, "scales": o.scales}
        if case["op"] == "rope":
            return hq.rope(st["desc"], st["x"], st["positions"], st["freqs"], st["gamma_q"], st["gamma_k"])
        desc, epilogue = st["desc"]
        return hq.adapters(desc, st["x"], st["a"], st["b"], st["ids"], scales=st["scales"], base=st["base"], epilogue=epilogue)
    if case["op"] == "rms_norm":
        return _plain_rms(case, st)
    return _plain_rope(case, st) if case["op"] == "rope" else _plain_adapters(case, st)


def _plain_rms(case, st):
    h = st["x"].float() if st["residual"] is None else st["x"].float() + st["residual"].float()
    rstd = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)
    out = {"h": h.to(st["x"].dtype) if "h" in case["outputs"] else None,
           "y": (h * rstd * st["gamma"]).to(st["x"].dtype) if "y" in case["outputs"] else None, "codes": None, "scales": None}
    if "q" in case["outputs"]:
        # a row's codes do not depend on its norm; a value next to a rounding border must not depend on the order
        # or the rounding of products, so they are decided in 64 bits
        v = st["x"].double() if st["residual"] is None else st["x"].double() + st["residual"].double()
        v = v * st["gamma"].double()
        s = v.abs().amax(1, keepdim=True) / 127.0
        out["codes"] = torch.where(s > 0, torch.round(v / s), torch.zeros_like(v)).to(torch.int8)
        out["scales"] = (s.float() * rstd).squeeze(1)
    return out


def _plain_rope(case, st):
    T, dim, q, k = case["T"], case["head_dim"], case["q_heads"], case["k_heads"]
    pairs = _pairs(case)
    half = sum(pairs)
    x = st["x"][:, : (q + k) * dim].float().reshape(T, q + k, dim)
    if case["norm"]:
        gamma = st["gamma_q"].expand(q, dim) if not k else torch.cat((st["gamma_q"].expand(q, dim), st["gamma_k"].expand(k, dim)))
        x = x / torch.sqrt(x.square().mean(2, keepdim=True) + 1e-6) * gamma
    axis = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).to(x.device)
    angle = st["positions"].double()[:, axis] * st["freqs"]  # in 64 bits: positions can be far
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    s = -s if case["inverse"] else s
    if case["halves"]:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), 2)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), 3).reshape(T, q + k, 2 * half)
    return torch.cat((turned, x[..., 2 * half:]), 2).reshape(T, (q + k) * dim).to(st["x"].dtype)


def _plain_adapters(case, st):
    T, k, n, r, count = case["T"], case["d_in"], case["d_out"], case["rank"], case["count"]
    u = (st["x"].float() @ st["a"].float().reshape(count * r, k).t()).reshape(T, count, r)
    mine = st["ids"][:, None] == torch.arange(count, device=u.device)[None, :]
    u = torch.where(mine[:, :, None], u * st["scales"][None, :, None], torch.zeros_like(u)).reshape(T, count * r)
    v = st["base"].float() + u @ st["b"].float().permute(0, 2, 1).reshape(count * r, n)
    if case["act"] == "silu":
        v = v / (1.0 + torch.exp(-v))
    if case["act"] == "gelu_tanh":
        v = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v.to(st["base"].dtype)


def work(case):
    size, T = 2 if case["dtype"] == "bf16" else 4, case["T"]
    if case["op"] == "rms_norm":
        values = 1 + case["residual"] + ("h" in case["outputs"]) + ("y" in case["outputs"])
        codes = T * case["C"] + 4.0 * T if "q" in case["outputs"] else 0.0
        return {"bytes": float(T * case["C"] * size * values + codes + 4 * case["C"]), "flops": 8.0 * T * case["C"]}
    if case["op"] == "rope":
        values = T * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        small = 4 * T * len(_pairs(case)) + 8 * sum(_pairs(case)) + (8 * case["head_dim"] if case["norm"] else 0)
        return {"bytes": float(2 * values * size + small), "flops": float(values * (7 if case["norm"] else 3))}
    k, n, r = case["d_in"], case["d_out"], case["rank"]
    used = min(case["count"], T)
    return {"bytes": float(size * (T * k + 2 * T * n + used * r * (k + n)) + 4 * T), "flops": 2.0 * T * r * (k + n)}


def exact(case, seed):
    """The definitions once more, in float64 and by other routes: norms by their lengths, rotations as products
    of complex numbers, adapters one by one."""
    st, T = prepare(case, seed), case["T"]
    if case["op"] == "rms_norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h = h + st["residual"].double()
        unit = h * (math.sqrt(case["C"]) / torch.sqrt((h * h).sum(1) + 1e-6 * case["C"]))[:, None]
        y = unit * st["gamma"].double()
        top = y.abs().max(1).values
        codes = (h * st["gamma"].double() * 127.0 / (h * st["gamma"].double()).abs().max(1).values.clamp_min(1e-300)[:, None])
        return {"h": h if "h" in case["outputs"] else None, "y": y if "y" in case["outputs"] else None,
                "codes": codes.round().to(torch.int8) if "q" in case["outputs"] else None,
                "scales": top / 127.0 if "q" in case["outputs"] else None}
    if case["op"] == "rope":
        q, k, dim, pairs = case["q_heads"], case["k_heads"], case["head_dim"], _pairs(case)
        half = sum(pairs)
        x = st["x"].double().view(T, -1, dim)[:, : q + k].clone()
        if case["norm"]:
            x *= math.sqrt(dim) / torch.sqrt((x * x).sum(2, keepdim=True) + 1e-6 * dim)
            x[:, :q] *= st["gamma_q"].double()
            if k:
                x[:, q:] *= st["gamma_k"].double()
        column = [a for a, p in enumerate(pairs) for _ in range(p)]
        angle = torch.stack([st["positions"][:, a].double() * st["freqs"][i] for i, a in enumerate(column)], 1)
        turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[:, None, :]
        if case["halves"]:
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
            x[..., :half], x[..., half:2 * half] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., : 2 * half].reshape(T, q + k, half, 2).contiguous()) * turn
            x[..., : 2 * half] = torch.view_as_real(z).reshape(T, q + k, 2 * half)
        return x.reshape(T, (q + k) * dim)
    v = st["base"].double()
    for a in range(case["count"]):
        rows = (st["ids"] == a).nonzero().squeeze(1)
        if rows.numel():
            u = torch.mm(st["x"][rows].double(), st["a"][a].double().t().contiguous())
            v[rows] += st["scales"][a].double() * torch.mm(u, st["b"][a].double().t().contiguous())
    if case["act"] == "silu":
        v = v * torch.sigmoid(v)
    if case["act"] == "gelu_tanh":
        v = v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v
