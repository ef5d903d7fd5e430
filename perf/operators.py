"""The operators that stand around a low-bit layer, as they are measured.

* ``linear``: Y = R + g * phi(X W^T + b), the layers of a diffusion transformer or a learned image
  codec that stay in 16 or 32 bits (embedders, modulation tables, caption projection, last layer,
  1x1 convolutions), with the activation phi, the gate g (one row per sample) and the residual R in
  the product's epilogue.
* ``quant_linear``: the same epilogue on the rotated-and-centred low-bit layer.
* ``group_norm``: group norm over channels-last data with an activation behind it.

Each has a plain form in elementary torch operations (``own`` false) and the framework's call
(``own`` true). Inputs come from the seed alone.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _linear(name, T, d_in, d_out, dtype, act, bias=True, residual=False, samples=0):
    return {"name": name, "op": "linear", "T": T, "d_in": d_in, "d_out": d_out, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "samples": samples}


def _quant(name, T, d_in, d_out, block, bits, x_dtype, act, smooth, center, residual=False, samples=0):
    return {"name": name, "op": "quant_linear", "T": T, "d_in": d_in, "d_out": d_out, "block": block, "bits": bits,
            "dtype": x_dtype, "act": act, "smooth": smooth, "center": center, "residual": residual, "samples": samples}


def _norm(name, samples, positions, channels, groups, dtype, act):
    return {"name": name, "op": "group_norm", "samples": samples, "positions": positions, "channels": channels,
            "groups": groups, "dtype": dtype, "act": act}


def listed():
    return [
        # first layer of the timestep embedder, one image: nothing but latency
        _linear("timestep_embed", 1, 256, 1152, "bf16", "silu"),
        # the modulation table of a block stack for two samples: six vectors of 1152 each
        _linear("adaln_table", 2, 1152, 6912, "bf16", "none"),
        # caption projection: 300 text tokens of a 4096-wide encoder
        _linear("caption_proj", 300, 4096, 1152, "bf16", "gelu_tanh"),
        # MLP output of a block left in 16 bits, two images of 4096 tokens, gated into the residual stream
        _linear("mlp_out_gated", 8192, 4608, 1152, "bf16", "none", residual=True, samples=2),
        # the square projection's shape in 16 bits, the largest product
        _linear("square4k_gelu", 8192, 4096, 4096, "bf16", "gelu"),
        # sizes that fill no tile: an odd token count, widths that are multiples of 8 only
        _linear("ragged", 1037, 1160, 2312, "bf16", "relu", residual=True),
        # a 1x1 convolution of the image codec in 32 bits with its skip connection, 8 latents of 32 x 48
        _linear("lic_conv_f32", 12288, 256, 256, "f32", "silu", residual=True),
        # the low-bit MLP input layer of a block with its GELU
        _quant("dit_fc1_w4a4_gelu", 8192, 1152, 4608, 128, 4, "bf16", "gelu_tanh", True, True),
        # the low-bit MLP output layer, gated into the residual stream, a ragged token count over three samples
        _quant("dit_fc2_w4a4_gated", 4353, 4608, 1152, 512, 4, "bf16", "none", True, True, residual=True, samples=3),
        # a small odd block of a U-shaped denoiser: ten channels per group
        _norm("unet_ragged", 3, 77, 320, 32, "bf16", "silu"),
        # the image codec's latents, before its 1x1 convolution
        _norm("lic_f32", 8, 1536, 256, 32, "f32", "silu"),
        # last stage of a latent decoder, one 512 x 512 image
        _norm("decoder_512", 1, 262144, 128, 32, "bf16", "silu"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step + 0.5) * step)


def draw(rng):
    op = rng.choice(("linear", "linear", "quant_linear", "group_norm", "group_norm"))
    act = rng.choice(ACTS)
    if op == "linear":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        while True:
            T, k, n = _log(rng, 1, 12288), _log(rng, 16, 6144, 8), _log(rng, 8, 8192, 8)
            if 2.0 * T * k * n <= (2.0e11 if dtype == "bf16" else 2.0e10) and T >= 1:
                break
        residual = rng.random() < 0.5
        samples = rng.choice((0, 1, 2, 3)) if residual else 0
        return {"op": op, "T": T, "d_in": k, "d_out": n, "dtype": dtype, "act": act, "bias": rng.random() < 0.8,
                "residual": residual, "samples": min(samples, T)}
    if op == "quant_linear":
        bits = rng.choice((4, 4, 8))
        while True:
            T, n = _log(rng, 1, 8192), _log(rng, 64, 6144, 8)
            k = rng.choice((128, 256, 384, 640, 1152, 1280, 2048, 2560, 4096, 4608))
            if 2.0 * T * k * n <= 1.0e11 and T >= 1:
                break
        block = 1 << rng.randrange(3, (k & -k).bit_length())
        residual = rng.random() < 0.5
        return {"op": op, "T": T, "d_in": k, "d_out": n, "block": block, "bits": bits,
                "dtype": rng.choice(("bf16", "bf16", "f32")), "act": act, "smooth": rng.random() < 0.6,
                "center": rng.random() < 0.6, "residual": residual, "samples": min(T, rng.choice((0, 1, 2, 5))) if residual else 0}
    while True:
        groups = rng.choice((1, 4, 8, 16, 32, 32))
        channels = groups * _log(rng, 1, 64)
        samples, positions = _log(rng, 1, 64), _log(rng, 1, 65536)
        if channels % 8 == 0 and 16 <= channels <= 2048 and samples * positions * channels <= 30_000_000:
            break
    return {"op": op, "samples": samples, "positions": positions, "channels": channels, "groups": groups,
            "dtype": rng.choice(("bf16", "f32")), "act": rng.choice(("none", "silu", "silu", "gelu", "relu"))}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _hadamard(order, dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < order:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h / math.sqrt(order)


def _rotate(x, block):
    """x [R, K] times the block-diagonal normalised Hadamard matrix, in x's type."""
    return (x.reshape(-1, block) @ _hadamard(block, x.dtype)).reshape(x.shape)


def _gate_rows(case):
    """Tokens per sample: the last sample may be shorter."""
    return -(-case["T"] // case["samples"]) if case["samples"] else 0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "group_norm":
        s, p, c = case["samples"], case["positions"], case["channels"]
        # channels of a feature map have means and widths of their own
        mean, width = _randn(g, c), torch.exp(0.5 * _randn(g, c))
        st["x"] = (_randn(g, s, p, c) * width + mean).to(DTYPES[case["dtype"]])
        st["gamma"], st["beta"] = 1.0 + 0.2 * _randn(g, c), 0.2 * _randn(g, c)
    else:
        T, k, n, dt = case["T"], case["d_in"], case["d_out"], DTYPES[case["dtype"]]
        x = _randn(g, T, k)
        if case["op"] == "quant_linear":  # one channel in a hundred is an outlier
            far = torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")
            x[:, far] *= 30.0
            st["bias"] = 0.01 * _randn(g, n)
            y_dt = torch.bfloat16
        else:
            st["bias"] = 0.1 * _randn(g, n) if case["bias"] else None
            y_dt = dt
        st["x"], st["w"] = x.to(dt), (_randn(g, n, k) / math.sqrt(k)).to(dt)
        st["residual"] = _randn(g, T, n).to(y_dt) if case["residual"] else None
        st["gate"] = (0.5 * _randn(g, case["samples"], n)).to(y_dt) if case["samples"] else None
        if case["op"] == "quant_linear":
            w = st["w"].double()
            if case["smooth"]:
                top_x, top_w = st["x"].float().abs().amax(0), st["w"].float().abs().amax(0)
                st["sigma"] = torch.sqrt(top_x.clamp_min(1e-5) / top_w.clamp_min(1e-5))
                w = w * st["sigma"].double()
            w = _rotate(w, case["block"])
            q = float(2 ** (case["bits"] - 1) - 1)
            s_w = w.abs().amax(1, keepdim=True) / q
            # the weights of the plain form, laid out once: codes, scales and column sums
            st["w_codes"] = torch.round(w / s_w).clamp(-q, q).float()
            st["w_scale"], st["w_sum"] = s_w.squeeze(1).float(), w.sum(1).float()
    if own:
        st["plan"] = _plan(case, st)
    return st


def _plan(case, st):
    """What a program of the framework keeps for the layer: the descriptor and, for a low-bit layer, the prepared weights."""
    import hadamard_rotated_bit_amd as hq
    dt = {"f32": hq.F32, "bf16": hq.BF16}[case["dtype"]]
    act = {"none": hq.HQ_ACT_NONE, "relu": hq.HQ_ACT_RELU, "silu": hq.HQ_ACT_SILU, "gelu": hq.HQ_ACT_GELU,
           "gelu_tanh": hq.HQ_ACT_GELU_TANH}[case["act"]]
    if case["op"] == "group_norm":
        return {"desc": hq.NormDesc(case["channels"], case["groups"], eps=1e-5, act=act, x_dtype=dt, y_dtype=dt)}
    epi = hq.Epilogue(act=act, residual=st["residual"], gate=st["gate"], gate_rows=_gate_rows(case))
    if case["op"] == "linear":
        return {"desc": hq.LinearDesc(case["d_in"], case["d_out"], x_dtype=dt, w_dtype=dt, y_dtype=dt), "epi": epi}
    desc = hq.Desc(case["d_in"], case["d_out"], case["block"], case["bits"], case["bits"], case["center"],
                   case["smooth"], 0, dt, dt, hq.BF16)
    return {"desc": desc, "epi": epi, "weights": hq.prepare(desc, st["w"], st["bias"], st.get("sigma"))}


def _act(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _finish(v, st, case):
    """The epilogue on the product v [T, N] in 32 bits, rounded once to the output's type."""
    v = _act(v, case["act"])
    if st["gate"] is not None:
        rows = torch.div(torch.arange(case["T"], device=v.device), _gate_rows(case), rounding_mode="floor")
        v = v * st["gate"].float()[rows]
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(torch.bfloat16 if case["op"] == "quant_linear" else st["x"].dtype)


def run(st):
    case = st["case"]
    if own:
        import hadamard_rotated_bit_amd as hq
        p = st["plan"]
        if case["op"] == "linear":
            return hq.linear(p["desc"], st["x"], st["w"], st["bias"], epilogue=p["epi"])
        if case["op"] == "quant_linear":
            return hq.quant_linear(p["desc"], p["weights"], st["x"], epilogue=p["epi"])
        return hq.group_norm(p["desc"], st["x"], st["gamma"], st["beta"])
    if case["op"] == "linear":
        v = st["x"].float() @ st["w"].float().t()
        return _finish(v if st["bias"] is None else v + st["bias"], st, case)
    if case["op"] == "quant_linear":
        # up to the codes in 64 bits: a value next to a rounding border must not depend on the order of sums
        x = st["x"].double()
        if case["smooth"]:
            x = x / st["sigma"].double()
        x = _rotate(x, case["block"])
        mu = x.mean(1, keepdim=True) if case["center"] else torch.zeros_like(x[:, :1])
        x = x - mu
        q = float(2 ** (case["bits"] - 1) - 1)
        s_x = x.abs().amax(1, keepdim=True) / q
        codes = torch.where(s_x > 0, torch.round(x / s_x), torch.zeros_like(x)).clamp(-q, q).float()
        v = (codes @ st["w_codes"].t()) * s_x.float() * st["w_scale"] + st["bias"] + mu.float() * st["w_sum"]
        return _finish(v, st, case)
    x = st["x"].float().reshape(case["samples"], case["positions"], case["groups"], -1)
    x = x - x.mean((1, 3), keepdim=True)
    x = x / torch.sqrt(x.square().mean((1, 3), keepdim=True) + 1e-5)
    y = x.reshape(st["x"].shape) * st["gamma"] + st["beta"]
    return _act(y, case["act"]).to(st["x"].dtype)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "group_norm":
        n = case["samples"] * case["positions"] * case["channels"]
        return {"bytes": 2.0 * n * size + 8.0 * case["channels"], "flops": 8.0 * n}
    T, k, n = case["T"], case["d_in"], case["d_out"]
    out = 2 if case["op"] == "quant_linear" else size
    b = T * k * size + T * n * out * (2 if case["residual"] else 1) + 4.0 * n + case["samples"] * n * out
    if case["op"] == "quant_linear":
        # 4-bit codes held in 6 bits or 8-bit codes, a scale and a column sum for each output channel
        b += n * k * (0.75 if case["bits"] == 4 else 1.0) + 8.0 * n
    else:
        b += n * k * size
    return {"bytes": float(b), "flops": 2.0 * T * k * n}


def exact(case, seed):
    """The definitions once more, in float64 and by other routes: sums over an explicit Hadamard sign table,
    erfc and sigmoid forms of the activations, moments in place of differences."""
    st = prepare(case, seed)

    def phi(v):
        if case["act"] == "relu":
            return v.clamp_min(0.0)
        if case["act"] == "silu":
            return v * torch.sigmoid(v)
        if case["act"] == "gelu":
            return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
        if case["act"] == "gelu_tanh":
            return v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3))
        return v

    if case["op"] == "group_norm":
        s, p, c, n = case["samples"], case["positions"], case["channels"], case["groups"]
        per = c // n
        x = st["x"].double().view(s, p, n, per).permute(0, 2, 1, 3).reshape(s, n, p * per)
        m = x.sum(2, keepdim=True) / (p * per)
        v = (x * x).sum(2, keepdim=True) / (p * per) - m * m
        y = ((x - m) * torch.rsqrt(v.clamp_min(0.0) + 1e-5)).view(s, n, p, per).permute(0, 2, 1, 3).reshape(s, p, c)
        return phi(st["gamma"].double() * y + st["beta"].double())
    T, k, n = case["T"], case["d_in"], case["d_out"]
    x, w = st["x"].double(), st["w"].double()
    if case["op"] == "linear":
        v = torch.mm(x, w.t().contiguous())
        if st["bias"] is not None:
            v += st["bias"].double()
    else:
        b, q = case["block"], 2.0 ** (case["bits"] - 1) - 1.0
        i = torch.arange(b, device="cuda")
        bits = i[:, None] & i[None, :]
        odd = torch.zeros_like(bits)
        for k_bit in range(max(1, b.bit_length())):
            odd ^= (bits >> k_bit) & 1
        h = (1.0 - 2.0 * odd.double()) / math.sqrt(b)
        if case["smooth"]:
            x, w = x / st["sigma"].double(), w * st["sigma"].double()
        x, w = (torch.mm(t.view(-1, b), h).view(t.shape) for t in (x, w))
        mu = x.sum(1) / k if case["center"] else torch.zeros(T, dtype=torch.float64, device="cuda")
        x = x - mu[:, None]
        top_x, top_w = x.abs().max(1).values / q, w.abs().max(1).values / q
        codes_x = torch.round(x / top_x.clamp_min(1e-300)[:, None])
        codes_w = torch.round(w / top_w.clamp_min(1e-300)[:, None])
        v = torch.mm(codes_x, codes_w.t().contiguous()) * top_x[:, None] * top_w[None, :]
        v += st["bias"].double() + mu[:, None] * w.sum(1)[None, :]
    v = phi(v)
    if st["gate"] is not None:
        v = v * torch.repeat_interleave(st["gate"].double(), _gate_rows(case), 0)[:T]
    if st["residual"] is not None:
        v = v + st["residual"].double()
    return v
