"""hadamard_rotated_bit_amd: the rotated-and-centred low-bit linear layer on MI355X.

A thin Python face over libhq (include/hq.h). Every step of the layer runs in
the library's HIP kernels; this module only checks tensors, allocates outputs
and workspaces with torch, and passes device pointers and the current stream.

    desc = Desc(d_in=1152, d_out=4608, block=128, a_bits=4, w_bits=4,
                center=True, smooth=True, x_dtype=BF16, w_dtype=BF16, y_dtype=BF16)
    amax = channel_absmax(desc, X_calib)
    sig = sigma(desc, amax, weight, alpha=0.5)
    prep = prepare(desc, weight, bias, sig)
    Y = quant_linear(desc, prep, X)
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from ._lib import (HQ_ACT_GELU, HQ_ACT_GELU_TANH, HQ_ACT_NONE, HQ_ACT_RELU, HQ_ACT_SILU,
                   HQ_CENTER_CHANNEL, HQ_CENTER_NONE, HQ_CENTER_TOKEN, HQ_CODES_E2M3,
                   HQ_CODES_I8, HQ_GEMM_AUTO, HQ_GEMM_I8, HQ_INT_ACT_GELU, HQ_INT_ACT_NONE,
                   HQ_INT_ACT_RELU, HQ_INT_ACT_SILU, HQ_INT_DH, HQ_INT_WH,
                   HQ_LINEAR_256X192, HQ_LINEAR_256X256, HQ_LINEAR_FEW, HQ_LINEAR_ROWS,
                   HQ_LINEAR_T32, HQ_LINEAR_T32X4, HQ_LINEAR_T64, HQ_LINEAR_T64X2,
                   HQ_LINEAR_T64X128, HQ_LINEAR_T128, HQ_LINEAR_T128W8, HQ_LINEAR_T128X2,
                   HQ_LINEAR_T128X192, HQ_NORM_BLOCK, HQ_NORM_CHUNKS, HQ_NORM_CHUNKS_JOINED,
                   HQ_NORM_ROWS, HQ_POS_F32, HQ_POS_I32, HQ_RMS_CODES, HQ_RMS_SUM, HQ_RMS_Y,
                   HQ_ROPE_HALVES, HQ_ROPE_MAX_AXES, HQ_ROPE_PAIRS, HqDesc, HqError,
                   HqLayout, check, load)

F32, BF16 = 0, 1
_TORCH = {F32: torch.float32, BF16: torch.bfloat16}
_NAME = {F32: "f32", BF16: "bf16"}


@dataclasses.dataclass(frozen=True)
class Desc:
    """Layer descriptor; mirrors hq_desc. ``center``: 0 / False none, 1 / True
    per-token mean, 2 per-channel mean over the call's tokens (HQ_CENTER_*).
    ``group``: 0 one scale per row, 64 one per row and 64-channel group."""
    d_in: int
    d_out: int
    block: int
    a_bits: int = 4
    w_bits: int = 4
    center: int = HQ_CENTER_TOKEN
    smooth: bool = False
    rank: int = 0
    x_dtype: int = F32
    w_dtype: int = F32
    y_dtype: int = F32
    gemm: int = HQ_GEMM_AUTO
    group: int = 0

    def __post_init__(self):
        raw = HqDesc(self.d_in, self.d_out, self.block, self.a_bits, self.w_bits,
                     int(self.center), int(self.smooth), self.rank, self.x_dtype,
                     self.w_dtype, self.y_dtype, self.gemm, self.group)
        object.__setattr__(self, "_raw", raw)
        object.__setattr__(self, "_ref", ctypes.byref(raw))

    def c(self) -> HqDesc:
        return self._raw

    def sx_shape(self, T: int) -> tuple:
        """Shape of the activation scales of T tokens: (T,), or (d_in / 64, T)
        with group-wise scales (group-major)."""
        return (self.d_in // self.group, T) if self.group else (T,)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def validate(desc: Desc) -> None:
    check(load().hq_validate(desc._ref))


def prepared_bytes(desc: Desc) -> int:
    n = load().hq_prepared_bytes(desc._ref)
    if n == 0:
        check(load().hq_validate(desc._ref))
    return n


def layout(desc: Desc) -> HqLayout:
    out = HqLayout()
    check(load().hq_prepared_layout_of(desc._ref, ctypes.byref(out)))
    return out


def workspace_bytes(desc: Desc, T: int) -> int:
    n = load().hq_workspace_bytes(desc._ref, T)
    if n == 0:
        check(load().hq_validate(desc._ref))
        if T < 0:
            raise HqError(_lib.HQ_ERR_INVALID_ARG, "T must be >= 0")
    return n


def code_format(desc: Desc) -> int:
    """HQ_CODES_I8 or HQ_CODES_E2M3 (see the code formats in include/hq.h)."""
    f = load().hq_code_format(desc._ref)
    if f < 0:
        check(f)
    return f


def code_bytes(desc: Desc, rows: int) -> int:
    """Bytes of a code matrix of `rows` rows in the descriptor's code format."""
    if rows < 0:
        raise HqError(_lib.HQ_ERR_INVALID_ARG, "rows must be >= 0")
    n = load().hq_code_bytes(desc._ref, rows)
    if n == 0 and rows > 0:
        check(load().hq_validate(desc._ref))
    return n


def _need_codes(t: torch.Tensor, name: str, desc: Desc, rows: int) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in (torch.uint8, torch.int8) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8/int8 code buffer")
    need = code_bytes(desc, rows)
    if t.numel() < need:
        raise ValueError(f"{name} holds {t.numel()} bytes, {need} needed for {rows} rows")


def channel_absmax(desc: Desc, X: torch.Tensor) -> torch.Tensor:
    """Per-input-channel max |X| over tokens (calibration statistic of HadaNorm Eq. (3))."""
    T = X.shape[0]
    _need(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    out = torch.empty(desc.d_in, dtype=torch.float32, device=X.device)
    check(load().hq_channel_absmax(desc._ref, _ptr(X), T, _ptr(out), _stream()))
    return out


def sigma(desc: Desc, act_absmax: torch.Tensor, weight: torch.Tensor, alpha: float) -> torch.Tensor:
    """Smoothing scales sigma_i = max|X_i|^alpha / max|W_i|^(1-alpha) (HadaNorm Eq. (3))."""
    _need(act_absmax, "act_absmax", torch.float32, (desc.d_in,))
    _need(weight, "weight", _TORCH[desc.w_dtype], (desc.d_out, desc.d_in))
    out = torch.empty(desc.d_in, dtype=torch.float32, device=weight.device)
    check(load().hq_sigma(desc._ref, _ptr(act_absmax), _ptr(weight),
                          ctypes.c_float(alpha), _ptr(out), _stream()))
    return out


def prepare(desc: Desc, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
            sigma: Optional[torch.Tensor] = None, L1: Optional[torch.Tensor] = None,
            L2: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Offline weight transform; returns the prepared blob (uint8 device tensor)."""
    wdt = _TORCH[desc.w_dtype]
    _need(weight, "weight", wdt, (desc.d_out, desc.d_in))
    if bias is not None:
        _need(bias, "bias", torch.float32, (desc.d_out,))
    if sigma is not None:
        _need(sigma, "sigma", torch.float32, (desc.d_in,))
    if L1 is not None:
        _need(L1, "L1", wdt, (desc.d_in, desc.rank))
    if L2 is not None:
        _need(L2, "L2", wdt, (desc.rank, desc.d_out))
    blob = torch.empty(prepared_bytes(desc), dtype=torch.uint8, device=weight.device)
    check(load().hq_prepare_weights(desc._ref, _ptr(weight), _ptr(bias),
                                    _ptr(sigma), _ptr(L1), _ptr(L2), _ptr(blob), _stream()))
    return blob


def check_prepared(desc: Desc, prepared: torch.Tensor) -> None:
    check(load().hq_check_prepared(desc._ref, _ptr(prepared), _stream()))


def quant_linear(desc: Desc, prepared: torch.Tensor, X: torch.Tensor,
                 out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 epilogue: Optional["Epilogue"] = None) -> torch.Tensor:
    """Y = the quantised layer applied to X [T, d_in]; with ``epilogue``
    (hq_quant_linear_epi) Y = residual + gate * phi(layer(X))."""
    if epilogue is not None:
        return _quant_linear_epi(desc, prepared, X, out, workspace, epilogue)
    T = X.shape[0]
    _need(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    if out is None:
        out = torch.empty(T, desc.d_out, dtype=_TORCH[desc.y_dtype], device=X.device)
    else:
        _need(out, "out", _TORCH[desc.y_dtype], (T, desc.d_out))
    if workspace is None:
        workspace = torch.empty(max(workspace_bytes(desc, T), 1), dtype=torch.uint8,
                                device=X.device)
    # the library checks the workspace size itself
    check(load().hq_quant_linear(desc._ref, _ptr(prepared), _ptr(X), T, _ptr(out),
                                 _ptr(workspace), workspace.numel(), _stream()))
    return out


NOALLOC_SCRATCH_BYTES = 32 << 20   # HQ_NOALLOC_SCRATCH_BYTES of include/hq.h


def quant_linear_noalloc(desc: Desc, prepared: torch.Tensor, X: torch.Tensor,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """quant_linear with the library's static per-GPU scratch array as the
    workspace (hq_quant_linear_noalloc): the call allocates nothing on the
    device besides ``out`` when it is not given. Calls that overlap on one
    GPU share that array and must not run concurrently."""
    T = X.shape[0]
    _need(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    if out is None:
        out = torch.empty(T, desc.d_out, dtype=_TORCH[desc.y_dtype], device=X.device)
    else:
        _need(out, "out", _TORCH[desc.y_dtype], (T, desc.d_out))
    check(load().hq_quant_linear_noalloc(desc._ref, _ptr(prepared), _ptr(X), T, _ptr(out),
                                         _stream()))
    return out


def _channel(desc: Desc) -> bool:
    return int(desc.center) == HQ_CENTER_CHANNEL


def channel_center(desc: Desc, prepared: torch.Tensor, X: torch.Tensor,
                   workspace: Optional[torch.Tensor] = None):
    """Per-channel centring statistics of X (center = 2): (mean [d_in] =
    mean_t(X), bias_eff [d_out_pad] = b + mean_t(X) W)."""
    T = X.shape[0]
    _need(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    mean = torch.empty(desc.d_in, dtype=torch.float32, device=X.device)
    bias_eff = torch.empty(layout(desc).d_out_pad, dtype=torch.float32, device=X.device)
    if workspace is None:
        workspace = torch.empty(max(workspace_bytes(desc, T), 1), dtype=torch.uint8,
                                device=X.device)
    check(load().hq_channel_center(desc._ref, _ptr(prepared), _ptr(X), T, _ptr(mean),
                                   _ptr(bias_eff), _ptr(workspace), workspace.numel(),
                                   _stream()))
    return mean, bias_eff


def channel_center_into(desc: Desc, prepared: torch.Tensor, X: torch.Tensor,
                        mean: torch.Tensor, bias_eff: torch.Tensor,
                        workspace: torch.Tensor) -> None:
    """channel_center writing into preallocated ``mean`` [d_in] and
    ``bias_eff`` [d_out_pad] (no allocation; e.g. under graph capture)."""
    T = X.shape[0]
    _need(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    _need(mean, "mean", torch.float32, (desc.d_in,))
    _need(bias_eff, "bias_eff", torch.float32, (layout(desc).d_out_pad,))
    check(load().hq_channel_center(desc._ref, _ptr(prepared), _ptr(X), T, _ptr(mean),
                                   _ptr(bias_eff), _ptr(workspace), workspace.numel(),
                                   _stream()))


def act_quantize(desc: Desc, prepared: torch.Tensor, X: torch.Tensor, out=None, mean=None,
                 workspace: Optional[torch.Tensor] = None):
    """Activation stage alone: (codes, s_x, mu [T], U [T, rank] or None); s_x
    has desc.sx_shape(T) ([T], or [d_in / 64, T] with group-wise scales).

    ``codes`` is a uint8 buffer of code_bytes(desc, T) bytes in the
    descriptor's code format. ``out`` may supply that tuple preallocated.
    For center = 2 the third entry is the per-channel mean [d_in] that was
    subtracted (``mean`` if given, else channel_center's). With ``workspace``
    (workspace_bytes(desc, T) bytes) the stage runs exactly as inside
    quant_linear (hq_act_quantize_ws: the two-pass low-rank projection);
    without it, hq_act_quantize (one pass, the same bits)."""
    T = X.shape[0]
    _need(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    dev = X.device
    chan = _channel(desc)
    if chan and mean is None:
        mean = channel_center(desc, prepared, X)[0]
    if out is None:
        codes = torch.empty(max(code_bytes(desc, T), 1), dtype=torch.uint8, device=dev)
        s_x = torch.empty(desc.sx_shape(T), dtype=torch.float32, device=dev)
        mu = mean if chan else torch.empty(T, dtype=torch.float32, device=dev)
        U = torch.empty(T, desc.rank, dtype=torch.float32, device=dev) if desc.rank else None
    else:
        codes, s_x, mu, U = out
        if chan:
            mu = mean
        _need_codes(codes, "codes", desc, T)
        _need(s_x, "s_x", torch.float32, desc.sx_shape(T))
        if desc.rank:
            _need(U, "U", torch.float32, (T, desc.rank))
    _need(mu, "mu", torch.float32, (desc.d_in,) if chan else (T,))
    if workspace is None:
        check(load().hq_act_quantize(desc._ref, _ptr(prepared), _ptr(X), T, _ptr(codes),
                                     _ptr(s_x), _ptr(mu), _ptr(U), _stream()))
    else:
        check(load().hq_act_quantize_ws(desc._ref, _ptr(prepared), _ptr(X), T, _ptr(codes),
                                        _ptr(s_x), _ptr(mu), _ptr(U), _ptr(workspace),
                                        workspace.numel(), _stream()))
    return codes, s_x, mu, U


def act_transform(desc: Desc, prepared: torch.Tensor, X: torch.Tensor, mean=None):
    """Float X~ (normalised H, centred) and mu, before quantisation (debug export).
    For center = 2 the second entry is the per-channel mean that was subtracted."""
    T = X.shape[0]
    _need(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    xt = torch.empty(T, desc.d_in, dtype=torch.float32, device=X.device)
    if _channel(desc):
        mu = mean if mean is not None else channel_center(desc, prepared, X)[0]
        _need(mu, "mean", torch.float32, (desc.d_in,))
    else:
        mu = torch.empty(T, dtype=torch.float32, device=X.device)
    check(load().hq_act_transform(desc._ref, _ptr(prepared), _ptr(X), T, _ptr(xt),
                                  _ptr(mu), _stream()))
    return xt, mu


def gemm_i32(desc: Desc, a_codes: torch.Tensor, w_codes: torch.Tensor, T: int,
             N: int) -> torch.Tensor:
    """int32 accumulators [T, N] of a_codes (T rows) . w_codes (N rows)^T, both
    code buffers in the descriptor's code format."""
    _need_codes(a_codes, "a_codes", desc, T)
    _need_codes(w_codes, "w_codes", desc, N)
    acc = torch.empty(T, N, dtype=torch.int32, device=a_codes.device)
    check(load().hq_gemm_i32(desc._ref, _ptr(a_codes), _ptr(w_codes), T, N, _ptr(acc),
                             _stream()))
    return acc


def gemm_dequant(desc: Desc, prepared: torch.Tensor, codes: torch.Tensor, s_x: torch.Tensor,
                 mu: torch.Tensor, U: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """GEMM + dequant epilogue alone, from act_quantize's outputs (T = the last
    dimension of s_x). For center = 2, ``mu`` is channel_center's bias_eff [d_out_pad]."""
    T = s_x.shape[-1]
    _need_codes(codes, "codes", desc, T)
    _need(s_x, "s_x", torch.float32, desc.sx_shape(T))
    _need(mu, "mu", torch.float32, (layout(desc).d_out_pad,) if _channel(desc) else (T,))
    if desc.rank:
        _need(U, "U", torch.float32, (T, desc.rank))
    Y = out if out is not None else torch.empty(T, desc.d_out, dtype=_TORCH[desc.y_dtype],
                                                device=codes.device)
    _need(Y, "out", _TORCH[desc.y_dtype], (T, desc.d_out))
    check(load().hq_gemm_dequant(desc._ref, _ptr(prepared), _ptr(codes), _ptr(s_x),
                                 _ptr(mu), _ptr(U), T, _ptr(Y), _stream()))
    return Y


def prepared_views(desc: Desc, prepared: torch.Tensor) -> dict:
    """Views of the arrays inside a prepared blob (for inspection and tests);
    w_codes is the raw code buffer of the d_out weight rows."""
    L = layout(desc)
    npad, d = L.d_out_pad, desc.d_in

    def view(off, n, dtype, shape):
        nbytes = n * torch.empty(0, dtype=dtype).element_size()
        return prepared[off:off + nbytes].view(dtype).view(*shape)

    out = {
        "w_codes": prepared[L.w_codes:L.w_codes + code_bytes(desc, desc.d_out)],
        "s_w": (view(L.w_scale, npad * (d // desc.group), torch.float32,
                     (d // desc.group, npad))[:, :desc.d_out] if desc.group
                else view(L.w_scale, npad, torch.float32, (npad,))[:desc.d_out]),
        "c": view(L.c, npad, torch.float32, (npad,))[:desc.d_out],
        "bias": view(L.bias, npad, torch.float32, (npad,))[:desc.d_out],
        "sigma_inv": view(L.sigma_inv, d, torch.float32, (d,)),
    }
    if _channel(desc):
        out["weight"] = view(L.weight, desc.d_out * d, _TORCH[desc.w_dtype], (desc.d_out, d))
    return out


# ---- epilogues and dense layers ---------------------------------------------

def _fits(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> None:
    """_need, and that ``t`` is on GPU ``device``; one expression when it is."""
    if (isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype
            and t.shape == shape and t.is_contiguous()):
        return
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, X on cuda:{device}")


def _gpu_of(X: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> int:
    """Checks X like _need; returns its GPU."""
    device = X.get_device() if isinstance(X, torch.Tensor) else -1
    if device < 0 or X.dtype is not dtype or X.shape != shape or not X.is_contiguous():
        _need(X, name, dtype, shape)
    return device


def _workspace_of(workspace: Optional[torch.Tensor], nbytes: int, X: torch.Tensor, device: int):
    """(tensor that keeps it alive, address, bytes) of a call's workspace,
    allocated when it is needed and not given (the library checks its size)."""
    if workspace is None:
        if not nbytes:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    elif workspace.get_device() != device:
        raise ValueError(f"workspace is on {workspace.device}, X on cuda:{device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.nbytes


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object (0.1 us instead
# of 1 us, a tenth of a small call) and the current device of an initialised
# runtime (a GPU tensor is at hand), where torch has the functions.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(device: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


@dataclasses.dataclass(frozen=True)
class Epilogue:
    """Y = residual + gate * phi(V) behind a layer's output V (hq_epilogue).
    ``act``: HQ_ACT_*; ``residual`` [T, d_out] (may be the call's ``out``);
    ``gate`` [samples, d_out], one row per ``gate_rows`` rows of Y (rows of
    the gate may be strided: one part of a modulation table)."""
    act: int = HQ_ACT_NONE
    residual: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    gate_rows: int = 0

    def __post_init__(self):
        if self.residual is None and self.gate is None:   # the same struct for every call
            raw = _lib.HqEpilogue(self.act, None, None, self.gate_rows, 0)
            object.__setattr__(self, "_ref", ctypes.byref(raw))

    def _c(self, T: int, d_out: int, dtype: torch.dtype, device: int):
        g, r, ld = self.gate, self.residual, 0
        if r is None and g is None:
            return self._ref
        if r is not None:
            _fits(r, "residual", dtype, (T, d_out), device)
        if g is not None:
            if not isinstance(g, torch.Tensor) or not g.is_cuda or g.dtype != dtype:
                raise ValueError(f"gate must be a CUDA (HIP) tensor of {dtype}")
            rows = -(-T // self.gate_rows) if self.gate_rows > 0 else 0
            if g.dim() != 2 or g.shape[1] != d_out or g.shape[0] < rows:
                raise ValueError(f"gate must have shape (>= {rows}, {d_out}), got {tuple(g.shape)}")
            if g.stride(1) != 1:
                raise ValueError("gate rows must be contiguous")
            if g.get_device() != device:
                raise ValueError(f"gate is on {g.device}, X on cuda:{device}")
            ld = g.stride(0) if g.shape[0] > 1 else d_out
        return ctypes.byref(_lib.HqEpilogue(self.act, _addr(r), _addr(g), self.gate_rows, ld))


def _need_prepared(desc: Desc, prepared: torch.Tensor, device: int) -> None:
    """``prepared`` is a blob of ``desc``'s size on GPU ``device`` (what it holds:
    check_prepared)."""
    if not isinstance(prepared, torch.Tensor) or not prepared.is_contiguous():
        raise ValueError("prepared must be a contiguous tensor")
    if prepared.get_device() != device:
        raise ValueError(f"prepared is on {prepared.device}, X on cuda:{device}")
    need = getattr(desc, "_blob_bytes", None)   # the descriptor's own: asked for once
    if need is None:
        need = prepared_bytes(desc)
        object.__setattr__(desc, "_blob_bytes", need)
    if prepared.nbytes < need:
        raise ValueError(f"prepared has {prepared.nbytes} bytes, {need} needed")


def _quant_linear_epi(desc, prepared, X, out, workspace, epilogue):
    T = X.shape[0]
    device = _gpu_of(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    if device != _current_gpu():   # kernels launch on the current device
        with torch.cuda.device(device):
            return _quant_linear_epi(desc, prepared, X, out, workspace, epilogue)
    ydt = _TORCH[desc.y_dtype]
    if out is None:
        out = torch.empty(T, desc.d_out, dtype=ydt, device=X.device)
    else:
        _fits(out, "out", ydt, (T, desc.d_out), device)
    _need_prepared(desc, prepared, device)
    ep = epilogue._c(T, desc.d_out, ydt, device)
    lib = load()
    ws, ws_addr, ws_bytes = _workspace_of(workspace, lib.hq_workspace_bytes(desc._ref, T), X, device)
    check(lib.hq_quant_linear_epi(desc._ref, prepared.data_ptr(), X.data_ptr(), T, ep,
                                  out.data_ptr(), ws_addr, ws_bytes, _stream_of(device)))
    return out


@dataclasses.dataclass(frozen=True)
class LinearDesc:
    """Dense-layer descriptor; mirrors hq_linear_desc (x_dtype = w_dtype)."""
    d_in: int
    d_out: int
    x_dtype: int = F32
    w_dtype: int = F32
    y_dtype: int = F32

    def __post_init__(self):
        raw = _lib.HqLinearDesc(self.d_in, self.d_out, self.x_dtype, self.w_dtype, self.y_dtype)
        object.__setattr__(self, "_raw", raw)
        object.__setattr__(self, "_ref", ctypes.byref(raw))


def linear_workspace_bytes(desc: LinearDesc, T: int) -> int:
    """Workspace bytes of linear for T rows (0 for most shapes)."""
    n = load().hq_linear_workspace_bytes(desc._ref, T)
    if n == 0:
        check(load().hq_linear_validate(desc._ref))
        if T < 0:
            raise HqError(_lib.HQ_ERR_INVALID_ARG, "T must be >= 0")
    return n


def linear_plan(desc: LinearDesc, T: int) -> _lib.HqLinearPlan:
    """How linear runs T rows (hq_linear_plan_of)."""
    out = _lib.HqLinearPlan()
    check(load().hq_linear_plan_of(desc._ref, T, ctypes.byref(out)))
    return out


def linear(desc: LinearDesc, X: torch.Tensor, weight: torch.Tensor,
           bias: Optional[torch.Tensor] = None, epilogue: Optional[Epilogue] = None,
           out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = residual + gate * phi(X weight^T + bias) for X [T, d_in] and weight
    [d_out, d_in], both bf16 or both fp32 (hq_linear): the layers that are not
    quantised. ``workspace`` (linear_workspace_bytes(desc, T) bytes) is
    allocated when it is needed and not given."""
    T = X.shape[0]
    xdt = _TORCH[desc.x_dtype]
    device = _gpu_of(X, "X", xdt, (T, desc.d_in))
    if device != _current_gpu():   # kernels launch on the current device
        with torch.cuda.device(device):
            return linear(desc, X, weight, bias, epilogue, out, workspace)
    _fits(weight, "weight", _TORCH[desc.w_dtype], (desc.d_out, desc.d_in), device)
    if bias is not None:
        _fits(bias, "bias", torch.float32, (desc.d_out,), device)
    ydt = _TORCH[desc.y_dtype]
    if out is None:
        out = torch.empty(T, desc.d_out, dtype=ydt, device=X.device)
    else:
        _fits(out, "out", ydt, (T, desc.d_out), device)
    ep = None if epilogue is None else epilogue._c(T, desc.d_out, ydt, device)
    lib = load()
    ws, ws_addr, ws_bytes = _workspace_of(
        workspace, lib.hq_linear_workspace_bytes(desc._ref, T), X, device)
    check(lib.hq_linear(desc._ref, X.data_ptr(), weight.data_ptr(), _addr(bias), T, ep,
                        out.data_ptr(), ws_addr, ws_bytes, _stream_of(device)))
    return out


@dataclasses.dataclass(frozen=True)
class NormDesc:
    """Group-norm descriptor; mirrors hq_norm_desc."""
    channels: int
    groups: int
    eps: float = 1e-5
    act: int = HQ_ACT_NONE
    x_dtype: int = F32
    y_dtype: int = F32

    def __post_init__(self):
        raw = _lib.HqNormDesc(self.channels, self.groups, self.act, self.x_dtype, self.y_dtype,
                              self.eps)
        object.__setattr__(self, "_raw", raw)
        object.__setattr__(self, "_ref", ctypes.byref(raw))


def group_norm_workspace_bytes(desc: NormDesc, samples: int, positions: int) -> int:
    """Workspace bytes of group_norm (0 where one launch does it)."""
    n = load().hq_group_norm_workspace_bytes(desc._ref, samples, positions)
    if n == 0:
        check(load().hq_norm_validate(desc._ref))
        if samples < 0 or positions < 0:
            raise HqError(_lib.HQ_ERR_INVALID_ARG, "samples and positions must be >= 0")
    return n


def group_norm_plan(desc: NormDesc, samples: int, positions: int) -> _lib.HqNormPlan:
    """How group_norm runs a call of this size (hq_group_norm_plan)."""
    out = _lib.HqNormPlan()
    check(load().hq_group_norm_plan(desc._ref, samples, positions, ctypes.byref(out)))
    return out


def group_norm(desc: NormDesc, X: torch.Tensor, gamma: Optional[torch.Tensor] = None,
               beta: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """phi(group norm) of channels-last X [samples, positions, channels]
    (hq_group_norm). ``out`` may be X itself when the types are the same;
    ``workspace`` (group_norm_workspace_bytes bytes) is allocated when it is
    needed and not given."""
    if X.dim() != 3:
        raise ValueError(f"X must be [samples, positions, channels], got {tuple(X.shape)}")
    S, P, C = X.shape[0], X.shape[1], desc.channels
    device = _gpu_of(X, "X", _TORCH[desc.x_dtype], (S, P, C))
    if device != _current_gpu():   # kernels launch on the current device
        with torch.cuda.device(device):
            return group_norm(desc, X, gamma, beta, out, workspace)
    if gamma is not None:
        _fits(gamma, "gamma", torch.float32, (C,), device)
    if beta is not None:
        _fits(beta, "beta", torch.float32, (C,), device)
    ydt = _TORCH[desc.y_dtype]
    if out is None:
        out = torch.empty(S, P, C, dtype=ydt, device=X.device)
    else:
        _fits(out, "out", ydt, (S, P, C), device)
    lib = load()
    ws, ws_addr, ws_bytes = _workspace_of(
        workspace, lib.hq_group_norm_workspace_bytes(desc._ref, S, P), X, device)
    check(lib.hq_group_norm(desc._ref, X.data_ptr(), _addr(gamma), _addr(beta), S, P,
                            out.data_ptr(), ws_addr, ws_bytes, _stream_of(device)))
    return out


# ---- RMS norm, rotary positions, adapters ------------------------------------

@dataclasses.dataclass(frozen=True)
class RmsNormDesc:
    """RMS-norm descriptor; mirrors hq_rms_desc. ``outputs``: a sum of HQ_RMS_Y
    (the norm), HQ_RMS_SUM (X + residual) and HQ_RMS_CODES (int8 codes of the norm
    with a scale per row)."""
    channels: int
    eps: float = 1e-6
    outputs: int = HQ_RMS_Y
    x_dtype: int = F32
    y_dtype: int = F32

    def __post_init__(self):
        raw = _lib.HqRmsDesc(self.channels, self.outputs, self.x_dtype, self.y_dtype, self.eps)
        object.__setattr__(self, "_raw", raw)
        object.__setattr__(self, "_ref", ctypes.byref(raw))


class RmsNorm(NamedTuple):
    """rms_norm's outputs; None for those the descriptor does not ask for."""
    y: Optional[torch.Tensor]
    h: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def rms_norm(desc: RmsNormDesc, X: torch.Tensor, gamma: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             sum_out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
             scales: Optional[torch.Tensor] = None) -> RmsNorm:
    """RMS norm of h = X + residual for X [T, channels] (hq_rms_norm): y = h gamma /
    sqrt(mean(h^2) + eps), h itself, and y as int8 ``codes`` [T, channels] with
    ``scales`` [T] (y ~ codes * scales), which gemm_dequant takes for a layer of
    block 1 and 8-bit activations. ``sum_out`` (h) and ``out`` (y) may be X or
    residual; outputs not given are allocated."""
    if X.dim() != 2:
        raise ValueError(f"X must be [T, channels], got {tuple(X.shape)}")
    shape, xdt = (X.shape[0], desc.channels), _TORCH[desc.x_dtype]
    device = _gpu_of(X, "X", xdt, shape)
    if device != _current_gpu():   # kernels launch on the current device
        with torch.cuda.device(device):
            return rms_norm(desc, X, gamma, residual, out, sum_out, codes, scales)
    if residual is not None:
        _fits(residual, "residual", xdt, shape, device)
    if gamma is not None:
        _fits(gamma, "gamma", torch.float32, (desc.channels,), device)
    ydt, want = _TORCH[desc.y_dtype], desc.outputs
    # outputs of X's type and shape are allocated like X: half a microsecond less each
    if want & HQ_RMS_Y:
        if out is None:
            out = torch.empty_like(X) if ydt is xdt else X.new_empty(shape, dtype=ydt)
        else:
            _fits(out, "out", ydt, shape, device)
    elif out is not None:
        raise ValueError("out is not among the descriptor's outputs")
    if want & HQ_RMS_SUM:
        if sum_out is None:
            sum_out = torch.empty_like(X)
        else:
            _fits(sum_out, "sum_out", xdt, shape, device)
    elif sum_out is not None:
        raise ValueError("sum_out is not among the descriptor's outputs")
    if want & HQ_RMS_CODES:
        if codes is None:
            codes = X.new_empty(shape, dtype=torch.int8)
        else:
            _fits(codes, "codes", torch.int8, shape, device)
        if scales is None:
            scales = X.new_empty(shape[:1], dtype=torch.float32)
        else:
            _fits(scales, "scales", torch.float32, shape[:1], device)
    elif codes is not None or scales is not None:
        raise ValueError("codes are not among the descriptor's outputs")
    check(load().hq_rms_norm(desc._ref, X.data_ptr(), _addr(residual), _addr(gamma), shape[0],
                             _addr(sum_out), _addr(out), _addr(codes), _addr(scales),
                             _stream_of(device)))
    return RmsNorm(out, sum_out, codes, scales)


@dataclasses.dataclass(frozen=True)
class RopeDesc:
    """Rotary-position descriptor; mirrors hq_rope_desc. ``pairs``: the rotated pairs
    of each axis; ``layout``: HQ_ROPE_PAIRS (neighbours) or HQ_ROPE_HALVES; ``norm``:
    an RMS norm of each head before its rotation; ``inverse``: the opposite rotation;
    ``pos_dtype``: HQ_POS_I32 or HQ_POS_F32."""
    q_heads: int
    k_heads: int
    head_dim: int
    pairs: Tuple[int, ...]
    layout: int = HQ_ROPE_PAIRS
    norm: bool = False
    eps: float = 1e-6
    inverse: bool = False
    pos_dtype: int = HQ_POS_I32
    x_dtype: int = F32
    y_dtype: int = F32

    def __post_init__(self):
        pairs = tuple(int(p) for p in self.pairs)
        if not 1 <= len(pairs) <= HQ_ROPE_MAX_AXES:
            raise ValueError(f"pairs must name 1 to {HQ_ROPE_MAX_AXES} axes, got {pairs}")
        object.__setattr__(self, "pairs", pairs)
        raw = _lib.HqRopeDesc(self.q_heads, self.k_heads, self.head_dim, len(pairs),
                              (ctypes.c_int32 * HQ_ROPE_MAX_AXES)(*pairs), self.layout,
                              int(self.norm), int(self.inverse), self.pos_dtype, self.x_dtype,
                              self.y_dtype, self.eps)
        object.__setattr__(self, "_raw", raw)
        object.__setattr__(self, "_ref", ctypes.byref(raw))


def rope_freqs(desc: RopeDesc, theta: float = 10000.0, per_axis: bool = True,
               device="cuda") -> torch.Tensor:
    """The usual frequencies of ``desc``'s pairs, float64 (rope takes any others as
    well): theta^(-i / p) for pair i of an axis of p pairs, or with ``per_axis``
    false theta^(-i / P) for pair i of all P (the axes share one sequence)."""
    total = sum(desc.pairs)
    axes = desc.pairs if per_axis else (total,)
    e = torch.cat([torch.arange(p, dtype=torch.float64) / max(p, 1) for p in axes])
    return torch.pow(torch.tensor(float(theta), dtype=torch.float64), -e).to(device)


def _rows_of(t: torch.Tensor, name: str, dtype: torch.dtype, T: int, width: int) -> int:
    """Checks a [T, >= width] tensor whose rows may be strided; returns its row pitch."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor of {dtype}")
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] < width:
        raise ValueError(f"{name} must have shape ({T}, >= {width}), got {tuple(t.shape)}")
    if t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return t.stride(0) if T > 1 else -(-t.shape[1] // 8) * 8


def rope(desc: RopeDesc, X: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
         gamma_q: Optional[torch.Tensor] = None, gamma_k: Optional[torch.Tensor] = None,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary positions on the q and k heads at the start of each row of X [T, >=
    (q_heads + k_heads) head_dim] (hq_rope), behind an RMS norm of each head with
    ``desc.norm``. ``positions`` [T, axes], ``freqs`` float64 (rope_freqs). X and
    ``out`` may have strided rows (a packed projection); ``out`` may be X itself: q and
    k are then turned in place. Returns ``out``, allocated as [T, (q_heads + k_heads)
    head_dim] when it is not given."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("X must be a tensor [T, channels]")
    T, width = X.shape[0], (desc.q_heads + desc.k_heads) * desc.head_dim
    ldx = _rows_of(X, "X", _TORCH[desc.x_dtype], T, width)
    device = X.get_device()
    if device != _current_gpu():   # kernels launch on the current device
        with torch.cuda.device(device):
            return rope(desc, X, positions, freqs, gamma_q, gamma_k, out)
    _fits(positions, "positions", torch.float32 if desc.pos_dtype == HQ_POS_F32 else torch.int32,
          (T, len(desc.pairs)), device)
    _fits(freqs, "freqs", torch.float64, (sum(desc.pairs),), device)
    for g, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        if g is not None:
            _fits(g, name, torch.float32, (desc.head_dim,), device)
    if out is None:
        out = X.new_empty((T, width), dtype=_TORCH[desc.y_dtype])
        ldy = width
    else:
        ldy = _rows_of(out, "out", _TORCH[desc.y_dtype], T, width)
        if out.get_device() != device:
            raise ValueError(f"out is on {out.device}, X on cuda:{device}")
    check(load().hq_rope(desc._ref, X.data_ptr(), ldx, positions.data_ptr(), freqs.data_ptr(),
                         _addr(gamma_q), _addr(gamma_k), T, out.data_ptr(), ldy,
                         _stream_of(device)))
    return out


@dataclasses.dataclass(frozen=True)
class AdapterDesc:
    """Descriptor of low-rank adapters beside a projection; mirrors hq_adapter_desc
    (x_dtype = w_dtype; ``rank`` the largest of the adapters)."""
    d_in: int
    d_out: int
    rank: int
    x_dtype: int = F32
    w_dtype: int = F32
    y_dtype: int = F32

    def __post_init__(self):
        raw = _lib.HqAdapterDesc(self.d_in, self.d_out, self.rank, self.x_dtype, self.w_dtype,
                                 self.y_dtype)
        object.__setattr__(self, "_raw", raw)
        object.__setattr__(self, "_ref", ctypes.byref(raw))


def adapters_workspace_bytes(desc: AdapterDesc, T: int) -> int:
    """Workspace bytes of adapters for T rows."""
    n = load().hq_adapters_workspace_bytes(desc._ref, T)
    if n == 0:
        check(load().hq_adapter_validate(desc._ref))
        if T < 0:
            raise HqError(_lib.HQ_ERR_INVALID_ARG, "T must be >= 0")
    return n


def adapters(desc: AdapterDesc, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
             ids: torch.Tensor, scales: Optional[torch.Tensor] = None,
             base: Optional[torch.Tensor] = None, epilogue: Optional[Epilogue] = None,
             out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = residual + gate * phi(base + scales[a] B_a (A_a X)) row by row, a = ids[row]
    (hq_adapters): the low-rank adapters of many requests beside a projection that gave
    ``base`` [T, d_out] (absent: zeros). X [T, d_in], A [count, rank, d_in], B [count,
    d_out, rank], ids int32 [T] (outside 0 .. count - 1: no adapter). ``out`` may be
    base itself; ``workspace`` (adapters_workspace_bytes(desc, T) bytes) is allocated
    when it is needed and not given. Calls of more than 512 rows do best with rows of
    one adapter next to each other; rows of many requests may go in a call of their own."""
    if X.dim() != 2:
        raise ValueError(f"X must be [T, d_in], got {tuple(X.shape)}")
    T, wdt, ydt = X.shape[0], _TORCH[desc.w_dtype], _TORCH[desc.y_dtype]
    device = _gpu_of(X, "X", _TORCH[desc.x_dtype], (T, desc.d_in))
    if device != _current_gpu():   # kernels launch on the current device
        with torch.cuda.device(device):
            return adapters(desc, X, A, B, ids, scales, base, epilogue, out, workspace)
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        raise ValueError("A must be [count, rank, d_in]")
    count = A.shape[0]
    _fits(A, "A", wdt, (count, desc.rank, desc.d_in), device)
    _fits(B, "B", wdt, (count, desc.d_out, desc.rank), device)
    _fits(ids, "ids", torch.int32, (T,), device)
    if scales is not None:
        _fits(scales, "scales", torch.float32, (count,), device)
    if base is not None:
        _fits(base, "base", ydt, (T, desc.d_out), device)
    if out is None:
        out = X.new_empty((T, desc.d_out), dtype=ydt) if base is None else torch.empty_like(base)
    else:
        _fits(out, "out", ydt, (T, desc.d_out), device)
    ep = None if epilogue is None else epilogue._c(T, desc.d_out, ydt, device)
    lib = load()
    ws, ws_addr, ws_bytes = _workspace_of(
        workspace, lib.hq_adapters_workspace_bytes(desc._ref, T), X, device)
    check(lib.hq_adapters(desc._ref, X.data_ptr(), A.data_ptr(), B.data_ptr(), count,
                          ids.data_ptr(), _addr(scales), _addr(base), T, ep, out.data_ptr(),
                          ws_addr, ws_bytes, _stream_of(device)))
    return out


# ---- integer-only DH / WH layers with integer requantisation ---------------

@dataclasses.dataclass(frozen=True)
class IntDesc:
    """Descriptor of an integer-only layer; mirrors hq_int_desc. ``side``
    HQ_INT_WH (weight transformed along its outputs by H of order ``block``)
    or HQ_INT_DH (along its inputs by H of order ``in_block``); ``block`` is
    the order of the output-side integer transform (before the activation),
    ``act`` the activation to the next layer (HQ_INT_ACT_*), ``post_block``
    the order of the transform after it (the next layer's H_in)."""
    d_in: int
    d_out: int
    block: int
    w_dtype: int = F32
    side: int = _lib.HQ_INT_WH
    in_block: int = 1
    act: int = _lib.HQ_INT_ACT_NONE
    post_block: int = 1

    @property
    def x_width(self) -> int:
        """Input codes per token (a padded DH input order takes in_block)."""
        pad = self.side == _lib.HQ_INT_DH and self.in_block > self.d_in
        return self.in_block if pad else self.d_in

    @property
    def acc_width(self) -> int:
        """Accumulator channels (a padded WH output order has block of them)."""
        pad = self.side == _lib.HQ_INT_WH and self.block > self.d_out
        return self.block if pad else self.d_out

    @property
    def out_width(self) -> int:
        """Output codes per token (a padded post order writes post_block)."""
        return self.post_block if self.post_block > self.d_out else self.d_out

    def __post_init__(self):
        raw = _lib.HqIntDesc(self.d_in, self.d_out, self.block, self.w_dtype, self.side,
                             self.in_block, self.act, self.post_block)
        object.__setattr__(self, "_raw", raw)
        object.__setattr__(self, "_ref", ctypes.byref(raw))


def int_layout(desc: IntDesc) -> "_lib.HqIntLayout":
    out = _lib.HqIntLayout()
    check(load().hq_int_prepared_layout_of(desc._ref, ctypes.byref(out)))
    return out


def int_workspace_bytes(desc: IntDesc, T: int) -> int:
    if T < 0:
        raise HqError(_lib.HQ_ERR_INVALID_ARG, "T must be >= 0")
    n = load().hq_int_workspace_bytes(desc._ref, T)
    if n == 0:
        check(load().hq_int_validate(desc._ref))
    return n


def int_prepare(desc: IntDesc, weight: torch.Tensor, bias: Optional[torch.Tensor], s_x: float,
                s_y: float, s_z: float = 0.0, s_u: float = 0.0) -> torch.Tensor:
    """Offline transform of an integer-only layer; returns the prepared blob.
    s_z, s_u: the int8 grids around a SiLU/GELU table (ignored otherwise)."""
    _need(weight, "weight", _TORCH[desc.w_dtype], (desc.d_out, desc.d_in))
    if bias is not None:
        _need(bias, "bias", torch.float32, (desc.d_out,))
    n = load().hq_int_prepared_bytes(desc._ref)
    if n == 0:
        check(load().hq_int_validate(desc._ref))
    blob = torch.empty(n, dtype=torch.uint8, device=weight.device)
    check(load().hq_int_prepare(desc._ref, _ptr(weight), _ptr(bias), ctypes.c_float(s_x),
                                ctypes.c_float(s_y), ctypes.c_float(s_z), ctypes.c_float(s_u),
                                _ptr(blob), _stream()))
    return blob


def int_linear(desc: IntDesc, prepared: torch.Tensor, x_codes: torch.Tensor,
               out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 output codes [T, out_width] of the layer for int8 input codes
    [T, x_width]."""
    T = x_codes.shape[0]
    _need(x_codes, "x_codes", torch.int8, (T, desc.x_width))
    y = out if out is not None else torch.empty(T, desc.out_width, dtype=torch.int8,
                                                device=x_codes.device)
    _need(y, "out", torch.int8, (T, desc.out_width))
    nws = int_workspace_bytes(desc, T)
    ws = workspace if workspace is not None else torch.empty(
        max(nws, 1), dtype=torch.uint8, device=x_codes.device)
    check(load().hq_int_linear(desc._ref, _ptr(prepared), _ptr(x_codes), T, _ptr(y), _ptr(ws),
                               ws.numel(), _stream()))
    return y


def int_requant(desc: IntDesc, prepared: torch.Tensor, acc: torch.Tensor) -> torch.Tensor:
    """Requantisation alone: int8 [T, out_width] from int32 products
    [T, acc_width] (no bias)."""
    T = acc.shape[0]
    _need(acc, "acc", torch.int32, (T, desc.acc_width))
    y = torch.empty(T, desc.out_width, dtype=torch.int8, device=acc.device)
    check(load().hq_int_requant(desc._ref, _ptr(prepared), _ptr(acc), T, _ptr(y), _stream()))
    return y


def int_views(desc: IntDesc, prepared: torch.Tensor) -> dict:
    """Views of the arrays inside an integer-layer prepared blob (for tests)."""
    L = int_layout(desc)
    npad, d, a = L.d_out_pad, desc.x_width, desc.acc_width

    def view(off, n, dtype, shape):
        nbytes = n * torch.empty(0, dtype=dtype).element_size()
        return prepared[off:off + nbytes].view(dtype).view(*shape)

    return {
        "w_codes": view(L.w_codes, npad * d, torch.int8, (npad, d))[:a],
        "s_w": view(L.w_scale, npad, torch.float32, (npad,))[:a],
        "b_int": view(L.b_int, npad, torch.int32, (npad,))[:a],
        "mult": view(L.mult, npad, torch.int32, (npad,))[:a],
        "shift": view(L.shift, 1, torch.int32, (1,)),
        "wbar": view(L.wbar, a * d, torch.float32, (a, d)),
        "lut": view(L.lut, 256, torch.int8, (256,)),
        "mult_in": view(L.mult_in, 1, torch.int32, (1,)),
        "shift_in": view(L.shift_in, 1, torch.int32, (1,)),
    }
