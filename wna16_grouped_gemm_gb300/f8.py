"""Routed experts in 8-bit floats (C ABI of ``include/wna16_moe_f8.h``).

    sort_tokens          tokens' rows, copied to the rows of their experts
    unsort_tokens        every token's rows back, weighted and added up
    unsort_tokens_grad   the gradient of that
    linear_f8            e4m3 rows times one block-scaled e4m3 weight
    grouped_linear_f8    rows in expert order times their experts' weights
    quantize_blocks_f8   weights to e4m3 with a scale per block of 128 x 128
    forward_f8           sort -> gate/up -> SwiGLU -> down -> unsort

As in ``block``: argument checks and marshalling only, CUDA tensors, the current stream (or
``stream``), outputs allocated unless they are passed in.  8-bit rows (q, scales) are those of
``quantize_q8``, ``add_rmsnorm_q8`` and ``swiglu_q8`` with float8_e4m3fn and groups of 128.

Nothing here takes part in autograd: outputs carry no graph, whatever the inputs require.  A program that trains
calls the gradients itself: unsort_tokens without weights for sort_tokens, unsort_tokens_grad for unsort_tokens, the
products with transposed weights for theirs with respect to the rows.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding, block
from .binding import _check
from .block import _matrix, _new

BLOCK = 128

_entries = None


def declare(lib) -> dict:
    """Declare the entry points of a loaded library; their addresses by name."""
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    entries = {}
    for name, args in (
            ("sort_tokens", [P, I64, P, I64, I64, I64, I, P, I, I64, I64, P, P, P, P, P]),
            ("unsort_tokens", [P, I64, P, P, P, I64, I64, I, I, P, P]),
            ("unsort_tokens_grad", [P, P, P, P, I64, I64, I, I64, I, P, P, P]),
            ("linear_f8", [P, P, P, P, P, P, I64, I64, I64, I, P, P, SZ, P]),
            ("grouped_linear_f8", [P, P, P, P, P, I64, I64, I64, I64, I, P, P, SZ, P]),
            ("quantize_blocks_f8", [P, I64, I64, I64, I64, I64, I64, I, P, P, P])):
        f = getattr(lib, "wna16_moe_" + name)
        f.argtypes, f.restype = args, I
        entries[name] = ctypes.cast(f, P).value
    return entries


def _load() -> dict:
    global _entries
    if _entries is None:
        block._load()
        _entries = declare(binding.load_library())
    return _entries


def sort_tokens(x, topk_ids, experts: int, *, scales=None, expert_begin: int = 0, rows=None, row_scales=None,
                offsets=None, inv=None, stream=None):
    """Rows in the order of their experts: (rows, row_scales, offsets, inv).

    topk_ids int32 [T, topk]; slot (t, j) has expert topk_ids[t][j] - expert_begin, and
    is left out unless that lies in [0, experts) (at most 1024).  inv int32 [T, topk] is the row of each
    slot (-1: left out), offsets int32 [experts + 1] the experts' first rows; within an expert
    rows are in slot order.  rows [T * topk, K] holds x[t] at each of its slots' rows, row_scales
    likewise for scales fp32 [T, groups] (None without them).  x is bf16, fp16, fp32, int8 or
    float8_e4m3fn [T, K], its rows may be strided; x=None: only offsets and inv.
    Rows from offsets[experts] on are left as they were.  The gradient with respect to x is
    unsort_tokens(drows, inv)."""
    entry = (_entries or _load())["sort_tokens"]
    if offsets is None or inv is None or (x is not None and rows is None) or (scales is not None and row_scales is None):
        T, topk = _matrix(topk_ids, "topk_ids")
        if not 0 < experts <= 1024:
            raise ValueError(f"experts={experts} must be in [1, 1024]")
        if offsets is None:
            offsets = _new((experts + 1,), torch.int32, topk_ids, stream)
        if inv is None:
            inv = _new((T, topk), torch.int32, topk_ids, stream)
        if x is not None and rows is None:
            rows = _new((T * topk, _matrix(x, "x")[1]), x.dtype, x, stream)
        if scales is not None and row_scales is None:
            row_scales = _new((T * topk, _matrix(scales, "scales")[1]), torch.float32, scales, stream)
    rc = block._host.sort_tokens(entry, x, scales, topk_ids, experts, expert_begin, rows, row_scales, offsets, inv, stream)
    if rc:
        _check(rc)
    return rows, row_scales, offsets, inv


def unsort_tokens(y, inv, weights=None, *, addend=None, out=None, stream=None):
    """out [T, K] = sum_j weights[t][j] * y[inv[t][j]] (+ addend), in fp32, rounded once.

    y [R, K] bf16, fp16 or fp32, inv int32 [T, topk] (rows outside [0, R) are left out), weights
    fp32 [T, topk] (None: all 1), addend [T, K] of y's type (out=addend adds in place)."""
    entry = (_entries or _load())["unsort_tokens"]
    if out is None:
        out = _new((_matrix(inv, "inv")[0], _matrix(y, "y")[1]), y.dtype, y, stream)
    rc = block._host.unsort_tokens(entry, y, inv, weights, addend, out, stream)
    if rc:
        _check(rc)
    return out


def unsort_tokens_grad(dout, inv, y=None, weights=None, *, dy=None, dweights=None, want_dy: bool = True, stream=None):
    """The gradient of unsort_tokens(y, inv, weights) at dout [T, K]: (dy, dweights).

    dy [R, K] of dout's type: weights[t][j] * dout[t] at row inv[t][j] (rows that no slot has are left
    as they were; R is y's or dy's rows, else T * topk); None with want_dy=False.
    dweights fp32 [T, topk]: the dot products of dout[t] and y[inv[t][j]], 0 for slots left out;
    None without y."""
    entry = (_entries or _load())["unsort_tokens_grad"]
    if dy is None and want_dy:
        T, topk = _matrix(inv, "inv")
        dy = _new((T * topk if y is None else _matrix(y, "y")[0], _matrix(dout, "dout")[1]), dout.dtype, dout, stream)
    if y is None and dweights is not None:
        raise ValueError("dweights without y")
    if y is not None and dweights is None:
        dweights = _new(_matrix(inv, "inv"), torch.float32, dout, stream)
    rc = block._host.unsort_tokens_grad(entry, dout, inv, y, weights, dy, dweights, stream)
    if rc:
        _check(rc)
    return dy, dweights


def linear_f8(xq, x_scales, wq, w_scales, *, bias=None, addend=None, dtype=torch.bfloat16, out=None, workspace=None,
              stream=None):
    """out [T, N] = (xq * x_scales) @ (wq * w_scales).T (+ bias) (+ addend), with fp32 sums.

    xq float8_e4m3fn [T, K], x_scales fp32 [T, K / 128], wq float8_e4m3fn [N, K], w_scales fp32
    [ceil(N / 128), K / 128] (a scale per block of 128 x 128), bias fp32 [N], addend [T, N] of the
    output's type (out=addend adds in place).  K is a multiple of 128.  workspace: uint8, at least 4
    bytes, gets the status word for read_status; may be left out.
    With wt, wt_scales = quantize_blocks_f8(w.t()), linear_f8(dq, d_scales, wt, wt_scales) is the gradient
    with respect to the rows' values (dq, d_scales: the output's gradient in 8 bits)."""
    entry = (_entries or _load())["linear_f8"]
    if out is None:
        out = _new((_matrix(xq, "xq")[0], _matrix(wq, "wq")[0]), dtype if addend is None else addend.dtype, xq, stream)
    rc = block._host.linear_f8(entry, xq, x_scales, wq, w_scales, bias, addend, out, workspace, stream)
    if rc:
        _check(rc)
    return out


def grouped_linear_f8(xq, x_scales, wq, w_scales, offsets, *, dtype=torch.bfloat16, out=None, workspace=None,
                      stream=None):
    """linear_f8 with a weight per expert: rows offsets[e] .. offsets[e + 1] - 1 of xq [R, K] take wq[e].

    wq float8_e4m3fn [E, N, K], w_scales fp32 [E, ceil(N / 128), K / 128], offsets int32 [E + 1] (sort_tokens').
    Rows of out [R, N] outside [offsets[0], offsets[E]) are left as they were."""
    entry = (_entries or _load())["grouped_linear_f8"]
    if out is None:
        if not isinstance(wq, torch.Tensor) or wq.dim() != 3:
            raise ValueError("wq must be a [E, N, K] tensor")
        out = _new((_matrix(xq, "xq")[0], wq.shape[1]), dtype, xq, stream)
    rc = block._host.grouped_linear_f8(entry, xq, x_scales, wq, w_scales, offsets, out, workspace, stream)
    if rc:
        _check(rc)
    return out


def quantize_blocks_f8(w, *, q=None, scales=None, stream=None):
    """(q, scales) of a weight [N, K] or of weights [E, N, K] (bf16, fp16 or fp32; rows or columns contiguous)
    in e4m3 with a scale per block of 128 x 128: q of w's shape, scales fp32 [(E,) ceil(N / 128), K / 128].
    Weights, and the rows or columns of one, lie behind one another, with or without gaps; interleaved ones are refused."""
    entry = (_entries or _load())["quantize_blocks_f8"]
    if q is None or scales is None:
        if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
            raise ValueError("w must be a tensor of 2 or 3 dims")
        if q is None:
            q = _new(tuple(w.shape), torch.float8_e4m3fn, w, stream)
        if scales is None:
            scales = _new((*w.shape[:-2], -(-w.shape[-2] // BLOCK), w.shape[-1] // BLOCK), torch.float32, w, stream)
    rc = block._host.quantize_blocks_f8(entry, w, q, scales, stream)
    if rc:
        _check(rc)
    return q, scales


def forward_f8(xq, x_scales, topk_ids, topk_weights, w13, w13_scales, w2, w2_scales, *, expert_begin: int = 0,
               swiglu_limit: float = 7.0, addend=None, dtype=torch.bfloat16, out=None, stream=None):
    """The routed experts in 8-bit floats: out [T, K] = sum_j topk_weights[t][j] * W2_e swiglu(W13_e x_t) (+ addend).

    xq float8_e4m3fn [T, K], x_scales fp32 [T, K / 128]; w13 [E, 2N, K] (gate rows, then up rows) and w2
    [E, K, N] as for grouped_linear_f8.  The experts of the weights are [expert_begin, expert_begin + E); slots of
    others add nothing.  The products are rounded to `dtype`, the SwiGLU's rows to e4m3 in groups of 128.
    Buffers are of T * topk rows, and the SwiGLU works on all of them, also where most slots are of other experts."""
    if not isinstance(w13, torch.Tensor) or w13.dim() != 3:
        raise ValueError("w13 must be a [E, 2N, K] tensor")
    rows, row_scales, offsets, inv = sort_tokens(xq, topk_ids, w13.shape[0], scales=x_scales, expert_begin=expert_begin,
                                                 stream=stream)
    gu = grouped_linear_f8(rows, row_scales, w13, w13_scales, offsets, dtype=dtype, stream=stream)
    hq, hs = block.swiglu_q8(gu, swiglu_limit=swiglu_limit, q_dtype=torch.float8_e4m3fn, group_size=BLOCK, stream=stream)
    y = grouped_linear_f8(hq, hs, w2, w2_scales, offsets, dtype=dtype, stream=stream)
    return unsort_tokens(y, inv, topk_weights, addend=addend, out=out, stream=stream)
