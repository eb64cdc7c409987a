"""The operators around the routed experts (C ABI of ``include/wna16_moe_block.h``)
and the MoE block that runs them together with the routed-expert forward.

    add_rmsnorm_q8   residual addition + RMS norm, rows in 16 and in 8 bits
    route_scored     expert choice: sigmoid / softmax scores, selection bias, groups
    linear_q8        8-bit integer product, a scale per token and per output channel
    swiglu_q8        clamped SwiGLU, rows in 8 bits
    quantize_q8, dequantize_q8   rows to 8 bits and back
    moe_block        norm -> router -> routed experts + shared expert

As in ``binding``: argument checks and marshalling only, every function takes
CUDA tensors, runs on the current stream (or ``stream``) and needs the built
library.  Outputs may be passed in (``q=``, ``scales=``, ``out=``, ...), as a
program does that keeps its buffers between steps; otherwise they are allocated.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import binding
from .binding import _check

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_Q_TYPES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_SCORES = {"sigmoid": 0, "softmax": 1}
_GROUP_SCORES = {"top2": 0, "max": 1}

_lib = None


def declare(lib):
    """Argument types of the block operators' entry points."""
    P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    for name, args in (
            ("add_rmsnorm_q8", [P, I64, P, I64, P, I, I64, I64, I, F, I, I, P, P, P, P, P]),
            ("swiglu_q8", [P, I64, I64, I64, I, F, I, I, P, P, P]),
            ("quantize_q8", [P, I64, I64, I64, I, I, I, P, P, P]),
            ("dequantize_q8", [P, P, I64, I64, I, I, I, P, P]),
            ("route_scored", [P, I64, P, I64, I64, I, I, I, I, I, I, I, F, P, P, P]),
            ("linear_q8", [P, P, P, P, P, P, I64, I64, I64, I, P, P, SZ, P])):
        f = getattr(lib, "wna16_moe_" + name)
        f.argtypes, f.restype = args, I
    lib.wna16_moe_linear_q8_workspace_size.argtypes = [I64, I64, I64]
    lib.wna16_moe_linear_q8_workspace_size.restype = SZ
    return lib


def _load():
    global _lib
    if _lib is None:
        _lib = declare(binding.load_library())
    return _lib


# The raw calls behind torch.cuda.current_device() and current_stream(): a tenth
# of their time, which counts where a decode step makes several small calls.
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _first(t, name: str, stream) -> tuple[int, int]:
    """(device, stream) of a call, from its first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != _device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_device()}")
    return dev, _raw_stream(dev) if stream is None else stream.cuda_stream


def _rows(t, dev: int, name: str, dtype=None) -> int:
    """The row distance of a 2-D tensor with contiguous rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if (t.dtype not in _TYPES) if dtype is None else (t.dtype is not dtype):
        raise TypeError(f"{name} must be {dtype or 'bfloat16, float16 or float32'}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(t.shape)}")
    ld, step = t.stride()
    rows, cols = t.shape
    if cols > 1 and step != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return ld if rows > 1 else max(cols, 1)


def _ptr(t, dev: int, dtype, shape, name: str) -> int:
    """The address of a contiguous tensor of this type and shape."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _new(shape, dtype, dev: int, stream):
    """An output, allocated on the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _q_outputs(T: int, K: int, q_dtype, group_size: int, q, scales, dev: int, stream):
    """(q, scales, their addresses, the format)."""
    if q is not None:
        q_dtype = q.dtype
    q_type = _Q_TYPES.get(q_dtype)
    if q_type is None:
        raise TypeError(f"8-bit rows are torch.int8 or torch.float8_e4m3fn, got {q_dtype}")
    groups = (T, K // group_size if group_size > 0 else 1)
    if q is None:
        q = _new((T, K), q_dtype, dev, stream)
    if scales is None:
        scales = _new(groups, torch.float32, dev, stream)
    return (q, scales, _ptr(q, dev, q_dtype, (T, K), "q"), _ptr(scales, dev, torch.float32, groups, "scales"), q_type)


def add_rmsnorm_q8(x, weight, residual=None, *, eps: float = 1e-6, q_dtype=torch.int8, group_size: int = 0,
                   want_norm: bool = False, want_q: bool = True, q=None, scales=None, residual_out=None, norm_out=None,
                   stream=None):
    """h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight.

    x, residual: bf16, fp16 or fp32 [T, K] (rows may be strided), weight [K] of
    that type or fp32.  Returns (q, scales, residual_out, norm_out): y in 8 bits
    (q_dtype int8 or float8_e4m3fn, one scale per row or per group_size values;
    None, None with want_q=False), h in x's type (None without a residual) and
    y in x's type (None unless want_norm or norm_out is given).
    residual_out=residual updates the residual in place."""
    dev, s = _first(x, "x", stream)
    ldx = _rows(x, dev, "x")
    shape = x.shape
    T, K = shape
    dtype = x.dtype
    ldr = r_ptr = ro_ptr = no_ptr = q_ptr = s_ptr = None
    if residual is not None:
        ldr = _rows(residual, dev, "residual", dtype)
        if residual.shape != shape:
            raise ValueError(f"residual must be {tuple(shape)}, got {tuple(residual.shape)}")
        r_ptr = residual.data_ptr()
        if residual_out is None:
            residual_out = _new(shape, dtype, dev, stream)
        ro_ptr = _ptr(residual_out, dev, dtype, shape, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    w_dtype = torch.float32 if isinstance(weight, torch.Tensor) and weight.dtype is torch.float32 else dtype
    w_ptr = _ptr(weight, dev, w_dtype, (K,), "weight")
    if norm_out is None and want_norm:
        norm_out = _new(shape, dtype, dev, stream)
    if norm_out is not None:
        no_ptr = _ptr(norm_out, dev, dtype, shape, "norm_out")
    q_type = 0
    if want_q:
        q, scales, q_ptr, s_ptr, q_type = _q_outputs(T, K, q_dtype, group_size, q, scales, dev, stream)
    elif q is not None or scales is not None:
        raise ValueError("q or scales with want_q=False")
    _check((_lib or _load()).wna16_moe_add_rmsnorm_q8(
        x.data_ptr(), ldx, r_ptr, ldr or 0, w_ptr, _TYPES[w_dtype], T, K, _TYPES[dtype], eps, q_type, group_size, q_ptr,
        s_ptr, ro_ptr, no_ptr, s))
    return q, scales, residual_out, norm_out


def swiglu_q8(gu, *, swiglu_limit: float = 7.0, q_dtype=torch.int8, group_size: int = 0, q=None, scales=None,
              stream=None):
    """(q, scales) of silu(min(g, L)) * clamp(u, -L, L) in 8 bits; gu [T, 2N]
    holds g in its first N columns and u in the others (bf16, fp16 or fp32)."""
    dev, s = _first(gu, "gu", stream)
    ld = _rows(gu, dev, "gu")
    T, N2 = gu.shape
    if N2 % 2:
        raise ValueError(f"gu must have an even number of columns, got {N2}")
    q, scales, q_ptr, s_ptr, q_type = _q_outputs(T, N2 // 2, q_dtype, group_size, q, scales, dev, stream)
    _check((_lib or _load()).wna16_moe_swiglu_q8(gu.data_ptr(), ld, T, N2 // 2, _TYPES[gu.dtype], swiglu_limit, q_type,
                                                 group_size, q_ptr, s_ptr, s))
    return q, scales


def quantize_q8(x, *, q_dtype=torch.int8, group_size: int = 0, q=None, scales=None, stream=None):
    """(q, scales) of the rows of x [T, K] in 8 bits (weights [N, K]: one scale
    per output channel, which linear_q8 takes)."""
    dev, s = _first(x, "x", stream)
    ld = _rows(x, dev, "x")
    T, K = x.shape
    q, scales, q_ptr, s_ptr, q_type = _q_outputs(T, K, q_dtype, group_size, q, scales, dev, stream)
    _check((_lib or _load()).wna16_moe_quantize_q8(x.data_ptr(), ld, T, K, _TYPES[x.dtype], q_type, group_size, q_ptr,
                                                   s_ptr, s))
    return q, scales


def dequantize_q8(q, scales, *, dtype=torch.bfloat16, out=None, stream=None):
    """The values code * scale of 8-bit rows q [T, K], scales [T, groups], in `dtype`."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _Q_TYPES:
        raise TypeError("q must be an int8 or float8_e4m3fn tensor")
    dev, s = _first(q, "q", stream)
    shape = q.shape
    if len(shape) != 2 or scales.dim() != 2:
        raise ValueError(f"q and scales must have 2 dims, got {tuple(shape)} and {tuple(scales.shape)}")
    T, K = shape
    groups = scales.shape[1]
    if groups < 1 or K % groups:
        raise ValueError(f"scales must be [{T}, groups] with groups dividing {K}, got {tuple(scales.shape)}")
    if out is None:
        out = _new(shape, dtype, dev, stream)
    type_ = _TYPES.get(out.dtype)
    if type_ is None:
        raise TypeError(f"values are bfloat16, float16 or float32, got {out.dtype}")
    _check((_lib or _load()).wna16_moe_dequantize_q8(
        _ptr(q, dev, q.dtype, shape, "q"), _ptr(scales, dev, torch.float32, (T, groups), "scales"), T, K,
        _Q_TYPES[q.dtype], K // groups if groups > 1 else 0, type_, _ptr(out, dev, out.dtype, shape, "out"), s))
    return out


def route_scored(logits, topk: int, *, score: str = "sigmoid", bias=None, groups: int = 1, topk_groups: int = 1,
                 group_score: str = "top2", renormalize: bool = True, scale: float = 1.0, ids=None, weights=None,
                 stream=None):
    """Expert choice: (topk_ids int32 [T, topk], topk_weights fp32 [T, topk]) from
    logits [T, E] (fp32, bf16 or fp16; rows may be strided).  Scores are
    sigmoid(logits) or softmax(logits); `bias` fp32 [E] is added for the choice
    only.  With groups > 1 the experts are chosen inside the topk_groups groups
    of largest group_score ("top2": sum of the two best, "max": the best).  The
    weights are the chosen scores, divided by their sum (renormalize), times scale."""
    dev, s = _first(logits, "logits", stream)
    ld = _rows(logits, dev, "logits")
    T, E = logits.shape
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if group_score not in _GROUP_SCORES:
        raise ValueError(f"group_score must be one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    if topk < 1:
        raise ValueError(f"topk={topk} must be positive")
    shape = (T, topk)
    if ids is None:
        ids = _new(shape, torch.int32, dev, stream)
    if weights is None:
        weights = _new(shape, torch.float32, dev, stream)
    _check((_lib or _load()).wna16_moe_route_scored(
        logits.data_ptr(), ld, None if bias is None else _ptr(bias, dev, torch.float32, (E,), "bias"), T, E,
        _TYPES[logits.dtype], _SCORES[score], groups, topk_groups, _GROUP_SCORES[group_score], topk,
        1 if renormalize else 0, scale, _ptr(ids, dev, torch.int32, shape, "ids"),
        _ptr(weights, dev, torch.float32, shape, "weights"), s))
    return ids, weights


def linear_q8_workspace_size(T: int, K: int, N: int) -> int:
    return int((_lib or _load()).wna16_moe_linear_q8_workspace_size(T, K, N))


def _scale_ptr(t, dev: int, n: int, name: str) -> int:
    """Address of n fp32 scales, [n] or [n, 1]."""
    return _ptr(t, dev, torch.float32, (n, 1) if isinstance(t, torch.Tensor) and t.dim() == 2 else (n,), name)


def linear_q8(xq, x_scales, wq, w_scales, *, bias=None, addend=None, dtype=torch.bfloat16, out=None, workspace=None,
              stream=None):
    """out [T, N] = (xq @ wq.T) * x_scales[:, None] * w_scales (+ bias) (+ addend).

    xq int8 [T, K], x_scales fp32 [T] or [T, 1], wq int8 [N, K], w_scales fp32
    [N] or [N, 1], bias fp32 [N], addend [T, N] of the output's type (out=addend
    adds in place).  workspace: uint8, at least linear_q8_workspace_size(T, K, N)
    bytes, holds the status word for read_status; may be left out."""
    dev, s = _first(xq, "xq", stream)
    if not isinstance(wq, torch.Tensor) or xq.dim() != 2 or wq.dim() != 2:
        raise ValueError("xq and wq must be matrices")
    T, K = xq.shape
    N = wq.shape[0]
    shape = (T, N)
    if out is None:
        out = _new(shape, dtype if addend is None else addend.dtype, dev, stream)
    dtype = out.dtype
    type_ = _TYPES.get(dtype)
    if type_ is None:
        raise TypeError(f"the output is bfloat16, float16 or float32, got {dtype}")
    lib = _lib or _load()
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel()
        ws_ptr = _ptr(workspace, dev, torch.uint8, (ws_bytes,), "workspace")
        need = lib.wna16_moe_linear_q8_workspace_size(T, K, N)
        if ws_bytes < need:   # (an empty tensor has no address to refuse)
            raise binding.Wna16Error(binding.ERR_WORKSPACE_TOO_SMALL, f"workspace has {ws_bytes} bytes, needs {need}")
    _check(lib.wna16_moe_linear_q8(
        _ptr(xq, dev, torch.int8, (T, K), "xq"), _scale_ptr(x_scales, dev, T, "x_scales"),
        _ptr(wq, dev, torch.int8, (N, K), "wq"), _scale_ptr(w_scales, dev, N, "w_scales"),
        None if bias is None else _ptr(bias, dev, torch.float32, (N,), "bias"),
        None if addend is None else _ptr(addend, dev, dtype, shape, "addend"), T, K, N, type_,
        _ptr(out, dev, dtype, shape, "out"), ws_ptr, ws_bytes, s))
    return out


@dataclasses.dataclass
class MoEBlockWeights:
    """Weights of one MoE block: norm, router, routed experts (WNA16) and shared expert (8 bits)."""
    norm: torch.Tensor              # [K], x's type or fp32
    gate: torch.Tensor              # [E, K], x's type: router
    gate_bias: torch.Tensor | None  # fp32 [E], for the choice only
    w13_packed: torch.Tensor        # routed experts, as for forward()
    w13_scales: torch.Tensor
    w2_packed: torch.Tensor
    w2_scales: torch.Tensor
    shared_w13: torch.Tensor        # int8 [2 Ns, K], gate rows then up rows
    shared_w13_scales: torch.Tensor
    shared_w2: torch.Tensor         # int8 [K, Ns]
    shared_w2_scales: torch.Tensor


def moe_block(x, residual, w: MoEBlockWeights, *, topk: int, bits: int, group_size: int, group_size_w2: int = 0,
              score: str = "sigmoid", groups: int = 1, topk_groups: int = 1, group_score: str = "top2",
              renormalize: bool = True, scale: float = 1.0, swiglu_limit: float = 7.0, eps: float = 1e-6):
    """One MoE block: (out, residual) with h = x + residual,
    out = routed(norm(h)) + shared(norm(h)), residual = h.

    The norm's 16-bit rows go to the router and the routed experts, its 8-bit
    rows to the shared expert, whose second product adds the routed output."""
    q, qs, residual, normed = add_rmsnorm_q8(x, w.norm, residual, eps=eps, want_norm=True)
    ids, weights = route_scored(normed @ w.gate.t(), topk, score=score, bias=w.gate_bias, groups=groups,
                                topk_groups=topk_groups, group_score=group_score, renormalize=renormalize, scale=scale)
    routed = binding.forward(normed, ids, weights, w.w13_packed, w.w13_scales, w.w2_packed, w.w2_scales, bits=bits,
                             group_size=group_size, group_size_w2=group_size_w2, swiglu_limit=swiglu_limit)
    gu = linear_q8(q, qs, w.shared_w13, w.shared_w13_scales, dtype=x.dtype)
    hq, hs = swiglu_q8(gu, swiglu_limit=swiglu_limit)
    return linear_q8(hq, hs, w.shared_w2, w.shared_w2_scales, addend=routed, out=routed), residual
