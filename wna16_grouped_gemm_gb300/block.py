"""The operators around the routed experts (C ABI of ``include/wna16_moe_block.h``)
and the MoE block that runs them together with the routed-expert forward.

    add_rmsnorm_q8   residual addition + RMS norm, rows in 16 and in 8 bits
    route_scored     expert choice: sigmoid / softmax scores, selection bias, groups
    linear_q8        8-bit integer product, a scale per token and per output channel
    swiglu_q8        clamped SwiGLU, rows in 8 bits
    quantize_q8, dequantize_q8   rows to 8 bits and back
    moe_block        norm -> router -> routed experts + shared expert

As in ``binding``: argument checks and marshalling only (in the compiled module
``_host``), every function takes CUDA tensors, runs on the current stream (or
``stream``) and needs the built library.  Outputs may be passed in (``q=``, ``scales=``, ``out=``, ...), as a
program does that keeps its buffers between steps; otherwise they are allocated.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import binding
from .binding import _check

_SCORES = {"sigmoid": 0, "softmax": 1}
_GROUP_SCORES = {"top2": 0, "max": 1}

_lib = None
_host = None


def declare(lib):
    """Declare the block operators' entry points of a loaded library and keep their addresses."""
    P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.block = {}
    for name, args in (
            ("add_rmsnorm_q8", [P, I64, P, I64, P, I, I64, I64, I, F, I, I, P, P, P, P, P]),
            ("swiglu_q8", [P, I64, I64, I64, I, F, I, I, P, P, P]),
            ("quantize_q8", [P, I64, I64, I64, I, I, I, P, P, P]),
            ("dequantize_q8", [P, P, I64, I64, I, I, I, P, P]),
            ("route_scored", [P, I64, P, I64, I64, I, I, I, I, I, I, I, F, P, P, P]),
            ("linear_q8", [P, P, P, P, P, P, I64, I64, I64, I, P, P, SZ, P])):
        f = getattr(lib, "wna16_moe_" + name)
        f.argtypes, f.restype = args, I
        lib.block[name] = ctypes.cast(f, P).value
    lib.wna16_moe_linear_q8_workspace_size.argtypes = [I64, I64, I64]
    lib.wna16_moe_linear_q8_workspace_size.restype = SZ
    return lib


def _load():
    """The library, and the module that checks arguments and calls it (raises if either was not built)."""
    global _lib, _host
    if _host is None:
        try:
            from . import _host as host
        except ImportError as e:
            raise RuntimeError("the module _host is missing: build it with wna16_grouped_gemm_gb300.build.build()") from e
        # the raw calls behind torch.cuda.current_device() and current_stream(): a tenth of their time
        host.setup((torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.float8_e4m3fn, torch.int32, torch.uint8),
                   torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
        _host = host
    if _lib is None:
        _lib = declare(binding.load_library())
    return _lib


def _new(shape, dtype, like, stream):
    """An output, allocated on the stream that writes it."""
    if not isinstance(like, torch.Tensor) or not like.is_cuda:
        raise TypeError("the inputs must be CUDA tensors")
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _new_q(x, K: int, q_dtype, group_size: int, q, scales, stream):
    """What is missing of (q, scales) for 8-bit rows of K values."""
    if q is None:
        if q_dtype not in (torch.int8, torch.float8_e4m3fn):
            raise TypeError(f"8-bit rows are torch.int8 or torch.float8_e4m3fn, got {q_dtype}")
        q = _new((x.shape[0], K), q_dtype, x, stream)
    if scales is None:
        scales = _new((x.shape[0], K // group_size if group_size > 0 else 1), torch.float32, x, stream)
    return q, scales


def _matrix(x, name: str):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(x.shape)}")
    return x.shape


def add_rmsnorm_q8(x, weight, residual=None, *, eps: float = 1e-6, q_dtype=torch.int8, group_size: int = 0,
                   want_norm: bool = False, want_q: bool = True, q=None, scales=None, residual_out=None, norm_out=None,
                   stream=None):
    """h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight.

    x, residual: bf16, fp16 or fp32 [T, K] (rows may be strided), weight [K] of
    that type or fp32.  Returns (q, scales, residual_out, norm_out): y in 8 bits
    (q_dtype int8 or float8_e4m3fn, one scale per row or per group_size values;
    None, None with want_q=False), h in x's type (without a residual, where h = x:
    None unless residual_out is given) and y in x's type (None unless want_norm
    or norm_out is given).
    residual_out=residual updates the residual in place."""
    lib = _lib or _load()
    if want_q:
        if q is None or scales is None:
            q, scales = _new_q(x, _matrix(x, "x")[1], q_dtype, group_size, q, scales, stream)
    elif q is not None or scales is not None:
        raise ValueError("q or scales with want_q=False")
    if residual is not None and residual_out is None:
        residual_out = _new(_matrix(x, "x"), x.dtype, x, stream)
    if norm_out is None and want_norm:
        norm_out = _new(_matrix(x, "x"), x.dtype, x, stream)
    rc = _host.add_rmsnorm_q8(lib.block["add_rmsnorm_q8"], x, weight, residual, residual_out, norm_out, q, scales, eps,
                              group_size, stream)
    if rc:
        _check(rc)
    return q, scales, residual_out, norm_out


def swiglu_q8(gu, *, swiglu_limit: float = 7.0, q_dtype=torch.int8, group_size: int = 0, q=None, scales=None,
              stream=None):
    """(q, scales) of silu(min(g, L)) * clamp(u, -L, L) in 8 bits; gu [T, 2N]
    holds g in its first N columns and u in the others (bf16, fp16 or fp32)."""
    lib = _lib or _load()
    if q is None or scales is None:
        q, scales = _new_q(gu, _matrix(gu, "gu")[1] // 2, q_dtype, group_size, q, scales, stream)
    rc = _host.swiglu_q8(lib.block["swiglu_q8"], gu, q, scales, swiglu_limit, group_size, stream)
    if rc:
        _check(rc)
    return q, scales


def quantize_q8(x, *, q_dtype=torch.int8, group_size: int = 0, q=None, scales=None, stream=None):
    """(q, scales) of the rows of x [T, K] in 8 bits (weights [N, K]: one scale
    per output channel, which linear_q8 takes)."""
    lib = _lib or _load()
    if q is None or scales is None:
        q, scales = _new_q(x, _matrix(x, "x")[1], q_dtype, group_size, q, scales, stream)
    rc = _host.quantize_q8(lib.block["quantize_q8"], x, q, scales, group_size, stream)
    if rc:
        _check(rc)
    return q, scales


def dequantize_q8(q, scales, *, dtype=torch.bfloat16, out=None, stream=None):
    """The values code * scale of 8-bit rows q [T, K], scales [T, groups], in `dtype`."""
    lib = _lib or _load()
    if out is None:
        if not isinstance(q, torch.Tensor) or q.dtype not in (torch.int8, torch.float8_e4m3fn):
            raise TypeError("q must be an int8 or float8_e4m3fn tensor")
        out = _new(_matrix(q, "q"), dtype, q, stream)
    rc = _host.dequantize_q8(lib.block["dequantize_q8"], q, scales, out, stream)
    if rc:
        _check(rc)
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
    lib = _lib or _load()
    s, g = _SCORES.get(score), _GROUP_SCORES.get(group_score)
    if s is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if g is None:
        raise ValueError(f"group_score must be one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    if ids is None or weights is None:
        if topk < 1:
            raise ValueError(f"topk={topk} must be positive")
        shape = (_matrix(logits, "logits")[0], topk)
        ids = _new(shape, torch.int32, logits, stream) if ids is None else ids
        weights = _new(shape, torch.float32, logits, stream) if weights is None else weights
    rc = _host.route_scored(lib.block["route_scored"], logits, bias, ids, weights, s, groups, topk_groups, g, topk,
                            1 if renormalize else 0, scale, stream)
    if rc:
        _check(rc)
    return ids, weights


def linear_q8_workspace_size(T: int, K: int, N: int) -> int:
    return int((_lib or _load()).wna16_moe_linear_q8_workspace_size(T, K, N))


def linear_q8(xq, x_scales, wq, w_scales, *, bias=None, addend=None, dtype=torch.bfloat16, out=None, workspace=None,
              stream=None):
    """out [T, N] = (xq @ wq.T) * x_scales[:, None] * w_scales (+ bias) (+ addend).

    xq int8 [T, K], x_scales fp32 [T] or [T, 1], wq int8 [N, K], w_scales fp32
    [N] or [N, 1], bias fp32 [N], addend [T, N] of the output's type (out=addend
    adds in place).  workspace: uint8, at least linear_q8_workspace_size(T, K, N)
    bytes, holds the status word for read_status; may be left out."""
    lib = _lib or _load()
    if out is None:
        out = _new((_matrix(xq, "xq")[0], _matrix(wq, "wq")[0]), dtype if addend is None else addend.dtype, xq, stream)
    if workspace is not None:
        need = lib.wna16_moe_linear_q8_workspace_size(xq.shape[0], xq.shape[1], wq.shape[0])
        if workspace.numel() < need:   # (an empty tensor has no address to refuse)
            raise binding.Wna16Error(binding.ERR_WORKSPACE_TOO_SMALL,
                                     f"workspace has {workspace.numel()} bytes, needs {need}")
    rc = _host.linear_q8(lib.block["linear_q8"], xq, x_scales, wq, w_scales, bias, addend, out, workspace, stream)
    if rc:
        _check(rc)
    return out


@dataclasses.dataclass
class MoEBlockWeights:
    """Weights of one MoE block: norm, router, routed experts (WNA16) and shared expert (8 bits)."""
    norm: torch.Tensor              # [K], bf16 or fp32
    gate: torch.Tensor              # [E, K] router: bf16 (logits rounded to bf16) or fp32 (fp32 logits)
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
    out = routed(norm(h)) + shared(norm(h)), residual = h (residual None, as
    before a first layer: h = x, which is returned itself).

    x and residual are bf16 [T, K] (what the routed experts take).  The norm's
    16-bit rows go to the router and the routed experts, its 8-bit rows to the
    shared expert, whose second product adds the routed output.  The choice of
    experts is exact for the logits that route_scored gets, which are a library
    product in the gate's type: with a bf16 gate they are rounded to bf16, and
    experts whose logits agree to 8 bits are taken by index; with an fp32 gate
    they are fp32."""
    q, qs, h, normed = add_rmsnorm_q8(x, w.norm, residual, eps=eps, want_norm=True)
    logits = normed.to(w.gate.dtype) @ w.gate.t()
    ids, weights = route_scored(logits, topk, score=score, bias=w.gate_bias, groups=groups,
                                topk_groups=topk_groups, group_score=group_score, renormalize=renormalize, scale=scale)
    routed = binding.forward(normed, ids, weights, w.w13_packed, w.w13_scales, w.w2_packed, w.w2_scales, bits=bits,
                             group_size=group_size, group_size_w2=group_size_w2, swiglu_limit=swiglu_limit)
    gu = linear_q8(q, qs, w.shared_w13, w.shared_w13_scales, dtype=x.dtype)
    hq, hs = swiglu_q8(gu, swiglu_limit=swiglu_limit)
    return linear_q8(hq, hs, w.shared_w2, w.shared_w2_scales, addend=routed, out=routed), x if residual is None else h
