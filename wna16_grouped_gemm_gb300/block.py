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
from .binding import _check, _need

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


def _rows(t, name: str, dtype=None):
    """A 2-D tensor whose rows are contiguous; returns its row distance."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if (t.dtype not in _TYPES) if dtype is None else (t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'bfloat16, float16 or float32'}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _out(t, shape: tuple, dtype, name: str, like, stream):
    """The output tensor `t`, checked, or a new one (on the stream that writes it)."""
    if t is None:
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=like.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=like.device)
    _need(t, dtype, name)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    _same_device(like, t, name)
    return t


def _same_device(x, t, name: str):
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, not on {x.device}")


def _stream(x, stream) -> int:
    dev = x.device.index
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return stream.cuda_stream if stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _q_outputs(x, T: int, K: int, q_dtype, group_size: int, q, scales, stream):
    if q is not None:
        q_dtype = q.dtype
    if q_dtype not in _Q_TYPES:
        raise TypeError(f"8-bit rows are torch.int8 or torch.float8_e4m3fn, got {q_dtype}")
    groups = K // group_size if group_size > 0 else 1
    return (_out(q, (T, K), q_dtype, "q", x, stream),
            _out(scales, (T, groups), torch.float32, "scales", x, stream), _Q_TYPES[q_dtype])


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
    ldx = _rows(x, "x")
    T, K = x.shape
    ldr = 0
    if residual is not None:
        ldr = _rows(residual, "residual", x.dtype)
        if residual.shape != x.shape:
            raise ValueError(f"residual must be {tuple(x.shape)}, got {tuple(residual.shape)}")
        _same_device(x, residual, "residual")
        residual_out = _out(residual_out, (T, K), x.dtype, "residual_out", x, stream)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"weight must be a tensor of {x.dtype} or float32")
    _need(weight, weight.dtype, "weight", 1)
    if weight.shape[0] != K:
        raise ValueError(f"weight must be [{K}], got {tuple(weight.shape)}")
    _same_device(x, weight, "weight")
    if want_norm or norm_out is not None:
        norm_out = _out(norm_out, (T, K), x.dtype, "norm_out", x, stream)
    q_type = 0
    if want_q:
        q, scales, q_type = _q_outputs(x, T, K, q_dtype, group_size, q, scales, stream)
    elif q is not None or scales is not None:
        raise ValueError("q or scales with want_q=False")
    s = _stream(x, stream)
    _check(_load().wna16_moe_add_rmsnorm_q8(
        x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, weight.data_ptr(),
        _TYPES[weight.dtype], T, K, _TYPES[x.dtype], eps, q_type, group_size, None if q is None else q.data_ptr(),
        None if scales is None else scales.data_ptr(), None if residual_out is None else residual_out.data_ptr(),
        None if norm_out is None else norm_out.data_ptr(), s))
    return q, scales, residual_out, norm_out


def swiglu_q8(gu, *, swiglu_limit: float = 7.0, q_dtype=torch.int8, group_size: int = 0, q=None, scales=None,
              stream=None):
    """(q, scales) of silu(min(g, L)) * clamp(u, -L, L) in 8 bits; gu [T, 2N]
    holds g in its first N columns and u in the others (bf16, fp16 or fp32)."""
    ld = _rows(gu, "gu")
    T, N2 = gu.shape
    if N2 % 2:
        raise ValueError(f"gu must have an even number of columns, got {N2}")
    q, scales, q_type = _q_outputs(gu, T, N2 // 2, q_dtype, group_size, q, scales, stream)
    s = _stream(gu, stream)
    _check(_load().wna16_moe_swiglu_q8(gu.data_ptr(), ld, T, N2 // 2, _TYPES[gu.dtype], swiglu_limit, q_type,
                                       group_size, q.data_ptr(), scales.data_ptr(), s))
    return q, scales


def quantize_q8(x, *, q_dtype=torch.int8, group_size: int = 0, q=None, scales=None, stream=None):
    """(q, scales) of the rows of x [T, K] in 8 bits (weights [N, K]: one scale
    per output channel, scales.view(N) for linear_q8)."""
    ld = _rows(x, "x")
    T, K = x.shape
    q, scales, q_type = _q_outputs(x, T, K, q_dtype, group_size, q, scales, stream)
    s = _stream(x, stream)
    _check(_load().wna16_moe_quantize_q8(x.data_ptr(), ld, T, K, _TYPES[x.dtype], q_type, group_size, q.data_ptr(),
                                         scales.data_ptr(), s))
    return q, scales


def dequantize_q8(q, scales, *, dtype=torch.bfloat16, out=None, stream=None):
    """The values code * scale of 8-bit rows q [T, K], scales [T, groups], in `dtype`."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _Q_TYPES:
        raise TypeError("q must be an int8 or float8_e4m3fn tensor")
    _need(q, q.dtype, "q", 2)
    _need(scales, torch.float32, "scales", 2)
    T, K = q.shape
    groups = scales.shape[1]
    if scales.shape[0] != T or groups < 1 or K % groups:
        raise ValueError(f"scales must be [{T}, groups] with groups dividing {K}, got {tuple(scales.shape)}")
    _same_device(q, scales, "scales")
    if out is not None:
        dtype = out.dtype
    if dtype not in _TYPES:
        raise TypeError(f"values are bfloat16, float16 or float32, got {dtype}")
    out = _out(out, (T, K), dtype, "out", q, stream)
    s = _stream(q, stream)
    _check(_load().wna16_moe_dequantize_q8(q.data_ptr(), scales.data_ptr(), T, K, _Q_TYPES[q.dtype],
                                           K // groups if groups > 1 else 0, _TYPES[dtype], out.data_ptr(), s))
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
    ld = _rows(logits, "logits")
    T, E = logits.shape
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if group_score not in _GROUP_SCORES:
        raise ValueError(f"group_score must be one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
        if bias.shape[0] != E:
            raise ValueError(f"bias must be [{E}], got {tuple(bias.shape)}")
        _same_device(logits, bias, "bias")
    if topk < 1:
        raise ValueError(f"topk={topk} must be positive")
    ids = _out(ids, (T, topk), torch.int32, "ids", logits, stream)
    weights = _out(weights, (T, topk), torch.float32, "weights", logits, stream)
    s = _stream(logits, stream)
    _check(_load().wna16_moe_route_scored(
        logits.data_ptr(), ld, None if bias is None else bias.data_ptr(), T, E, _TYPES[logits.dtype], _SCORES[score],
        groups, topk_groups, _GROUP_SCORES[group_score], topk, 1 if renormalize else 0, scale, ids.data_ptr(),
        weights.data_ptr(), s))
    return ids, weights


def linear_q8_workspace_size(T: int, K: int, N: int) -> int:
    return int(_load().wna16_moe_linear_q8_workspace_size(T, K, N))


def linear_q8(xq, x_scales, wq, w_scales, *, bias=None, addend=None, dtype=torch.bfloat16, out=None, workspace=None,
              stream=None):
    """out [T, N] = (xq @ wq.T) * x_scales[:, None] * w_scales (+ bias) (+ addend).

    xq int8 [T, K], x_scales fp32 [T] or [T, 1], wq int8 [N, K], w_scales fp32
    [N] or [N, 1], bias fp32 [N], addend [T, N] of the output's type (out=addend
    adds in place).  workspace: uint8, at least linear_q8_workspace_size(T, K, N)
    bytes, holds the status word for read_status; may be left out."""
    _need(xq, torch.int8, "xq", 2)
    _need(wq, torch.int8, "wq", 2)
    _need(x_scales, torch.float32, "x_scales")
    _need(w_scales, torch.float32, "w_scales")
    T, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError(f"wq must be [N, {K}], got {tuple(wq.shape)}")
    if x_scales.numel() != T or w_scales.numel() != N:
        raise ValueError(f"x_scales must hold {T} and w_scales {N} values, got {tuple(x_scales.shape)} and "
                         f"{tuple(w_scales.shape)}")
    if out is not None:
        dtype = out.dtype
    elif addend is not None:
        dtype = addend.dtype
    if dtype not in _TYPES:
        raise TypeError(f"the output is bfloat16, float16 or float32, got {dtype}")
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
        if bias.shape[0] != N:
            raise ValueError(f"bias must be [{N}], got {tuple(bias.shape)}")
    if addend is not None:
        _need(addend, dtype, "addend", 2)
        if tuple(addend.shape) != (T, N):
            raise ValueError(f"addend must be {(T, N)}, got {tuple(addend.shape)}")
    for t, name in ((wq, "wq"), (x_scales, "x_scales"), (w_scales, "w_scales"), (bias, "bias"), (addend, "addend")):
        if t is not None:
            _same_device(xq, t, name)
    out = _out(out, (T, N), dtype, "out", xq, stream)
    s = _stream(xq, stream)
    lib = _load()
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
        _same_device(xq, workspace, "workspace")
        need = lib.wna16_moe_linear_q8_workspace_size(T, K, N)
        if workspace.numel() < need:   # (an empty tensor has no address to refuse)
            raise binding.Wna16Error(binding.ERR_WORKSPACE_TOO_SMALL,
                                     f"workspace has {workspace.numel()} bytes, needs {need}")
    _check(lib.wna16_moe_linear_q8(
        xq.data_ptr(), x_scales.data_ptr(), wq.data_ptr(), w_scales.data_ptr(), None if bias is None else bias.data_ptr(),
        None if addend is None else addend.data_ptr(), T, K, N, _TYPES[dtype], out.data_ptr(),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(), s))
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
