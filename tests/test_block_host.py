"""Host-side checks of the operators around the routed experts, without a GPU:
every declared symbol is exported, bad arguments are refused before any CUDA
call (the pointers here are never dereferenced), empty batches do nothing."""
from __future__ import annotations

import ctypes
import math
import os
import re

import pytest
import torch

from wna16_grouped_gemm_gb300 import binding, block, build

HEADER = os.path.join(os.path.dirname(binding.HEADER), "wna16_moe_block.h")
P = [0x10000000 * (i + 1) for i in range(8)]   # far apart
INV, UNS, SMALL = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED, binding.ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    build.build()
    return block._load()


def _names():
    with open(HEADER) as f:
        return re.findall(r"WNA16_API\s+[\w\s\*]+?\b(wna16_\w+)\s*\(", f.read())


def test_every_declared_symbol_is_exported_by_both_builds(lib):
    names = _names()
    assert len(names) == 7, names
    build.build(debug=True)
    for b in (lib, binding.load_debug_library()):
        for n in names:
            assert hasattr(b, n), n


def _norm(lib, *, x=P[0], ldx=4096, residual=P[1], ldr=4096, weight=P[2], weight_type=0, T=4, K=4096, type=0, eps=1e-6,
          q_type=0, group=0, q=P[3], scales=P[4], residual_out=P[5], norm_out=P[6]):
    return lib.wna16_moe_add_rmsnorm_q8(x, ldx, residual, ldr, weight, weight_type, T, K, type, eps, q_type, group, q,
                                        scales, residual_out, norm_out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), UNS), (dict(type=-1), UNS), (dict(weight_type=1), UNS), (dict(weight_type=3), UNS),
    (dict(T=-1), INV), (dict(K=0), INV), (dict(K=32769, ldx=40000, ldr=40000), UNS), (dict(T=1 << 31), UNS),
    (dict(ldx=4095), INV), (dict(ldr=100), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(eps=math.inf), INV), (dict(q_type=2), UNS), (dict(group=16), UNS), (dict(group=512), UNS),
    (dict(group=96), UNS), (dict(group=-32), UNS), (dict(K=4000, group=128), UNS),
    (dict(q=None), INV), (dict(scales=None), INV), (dict(q=None, scales=None, norm_out=None), INV),
    (dict(x=None), INV), (dict(weight=None), INV), (dict(x=P[0] + 1), INV), (dict(residual=P[1] + 1), INV),
    (dict(weight=P[2] + 2, weight_type=2), INV), (dict(scales=P[4] + 2), INV), (dict(norm_out=P[6] + 1), INV),
    (dict(norm_out=P[0]), INV),                                    # norm_out over x
    (dict(residual_out=P[1] + 2), INV),                            # a shifted residual, not in place
    (dict(residual_out=P[1], ldr=8192), INV),                      # in place needs contiguous rows
    (dict(residual_out=P[6]), INV),                                # two outputs in one place
    (dict(q=P[4]), INV), (dict(q=P[2]), INV), (dict(scales=P[0] + 4), INV),
])
def test_norm_refuses(lib, kw, code):
    assert _norm(lib, **kw) == code
    assert lib.wna16_moe_last_error().decode() != ""


def _swiglu(lib, *, gu=P[0], ld=4096, T=4, N=2048, type=0, limit=7.0, q_type=0, group=0, q=P[3], scales=P[4]):
    return lib.wna16_moe_swiglu_q8(gu, ld, T, N, type, limit, q_type, group, q, scales, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=5), UNS), (dict(T=-1), INV), (dict(N=0), INV), (dict(N=40000, ld=80000), UNS), (dict(ld=4095), INV),
    (dict(limit=0.0), INV), (dict(limit=-1.0), INV), (dict(limit=math.nan), INV), (dict(q_type=7), UNS),
    (dict(group=100), UNS), (dict(gu=None), INV), (dict(q=None), INV), (dict(scales=None), INV),
    (dict(gu=P[0] + 1), INV), (dict(q=P[0] + 64), INV), (dict(scales=P[3]), INV),
])
def test_swiglu_refuses(lib, kw, code):
    assert _swiglu(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=9), UNS), (dict(K=-4), INV), (dict(ld=10), INV), (dict(group=33), UNS), (dict(x=None), INV),
    (dict(q=P[0]), INV),
])
def test_quantize_refuses(lib, kw, code):
    a = dict(x=P[0], ld=4096, T=4, K=4096, type=0, q_type=0, group=0, q=P[3], scales=P[4]) | kw
    assert lib.wna16_moe_quantize_q8(a["x"], a["ld"], a["T"], a["K"], a["type"], a["q_type"], a["group"], a["q"],
                                     a["scales"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=9), UNS), (dict(K=0), INV), (dict(group=7), UNS), (dict(q=None), INV), (dict(scales=None), INV),
    (dict(out=None), INV), (dict(out=P[0] + 2), INV), (dict(out=P[5] + 1), INV), (dict(q_type=3), UNS),
])
def test_dequantize_refuses(lib, kw, code):
    a = dict(q=P[0], scales=P[4], T=4, K=4096, q_type=0, group=0, type=0, out=P[5]) | kw
    assert lib.wna16_moe_dequantize_q8(a["q"], a["scales"], a["T"], a["K"], a["q_type"], a["group"], a["type"],
                                       a["out"], None) == code


def _route(lib, *, logits=P[0], ld=256, bias=P[1], T=4, E=256, type=2, score=0, groups=8, topk_groups=4, group_score=0,
           topk=8, renorm=1, scale=1.0, ids=P[3], weights=P[4]):
    return lib.wna16_moe_route_scored(logits, ld, bias, T, E, type, score, groups, topk_groups, group_score, topk,
                                      renorm, scale, ids, weights, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), UNS), (dict(T=-1), INV), (dict(E=0), INV), (dict(E=2048, ld=2048), UNS), (dict(ld=255), INV),
    (dict(score=2), UNS), (dict(group_score=2), UNS), (dict(groups=0), INV), (dict(groups=7), INV),
    (dict(groups=64), INV), (dict(topk_groups=0), INV), (dict(topk_groups=9), INV), (dict(topk=0), INV),
    (dict(topk=33), INV), (dict(topk_groups=1, groups=32, topk=9), INV), (dict(renorm=2), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(logits=None), INV), (dict(logits=P[0] + 2), INV),
    (dict(bias=P[1] + 2), INV), (dict(ids=None), INV), (dict(weights=None), INV), (dict(ids=P[4]), INV),
    (dict(weights=P[0]), INV),
])
def test_route_refuses(lib, kw, code):
    assert _route(lib, **kw) == code


def _linear(lib, *, xq=P[0], xs=P[1], wq=P[2], ws=P[3], bias=None, addend=None, T=64, K=4096, N=4096, type=0, out=P[5],
            workspace=P[6], nbytes=1 << 40):
    return lib.wna16_moe_linear_q8(xq, xs, wq, ws, bias, addend, T, K, N, type, out, workspace, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=4), UNS), (dict(T=-1), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(K=4088), UNS),
    (dict(K=65552), UNS), (dict(T=1 << 24), UNS), (dict(N=1 << 24), UNS), (dict(xq=None), INV), (dict(wq=None), INV),
    (dict(xs=None), INV), (dict(ws=None), INV), (dict(xq=P[0] + 8), INV), (dict(wq=P[2] + 4), INV),
    (dict(xs=P[1] + 2), INV), (dict(bias=P[4] + 1), INV), (dict(addend=P[4] + 1), INV), (dict(out=None), INV),
    (dict(out=P[5] + 1), INV), (dict(workspace=P[6] + 16), INV), (dict(nbytes=100), SMALL),
    (dict(out=P[0] + 4096), INV), (dict(out=P[2]), INV), (dict(addend=P[5] + 2), INV), (dict(workspace=P[2]), INV),
])
def test_linear_refuses(lib, kw, code):
    assert _linear(lib, **kw) == code
    assert lib.wna16_moe_last_error().decode() != ""


def test_empty_batches_do_nothing(lib):
    none = dict(x=None, weight=None, q=None, scales=None, residual=None, residual_out=None, norm_out=None)
    assert _norm(lib, T=0, **none) == 0
    assert _swiglu(lib, T=0, gu=None, q=None, scales=None) == 0
    assert lib.wna16_moe_quantize_q8(None, 4096, 0, 4096, 0, 0, 0, None, None, None) == 0
    assert lib.wna16_moe_dequantize_q8(None, None, 0, 4096, 0, 0, 0, None, None) == 0
    assert _route(lib, T=0, logits=None, bias=None, ids=None, weights=None) == 0
    assert _linear(lib, T=0, xq=None, xs=None, wq=None, ws=None, out=None, workspace=None, nbytes=0) == 0


def test_linear_workspace_size(lib):
    size = lib.wna16_moe_linear_q8_workspace_size
    assert size(1, 4096, 4096) == 0                                   # small batches need none
    assert size(2048, 4096, 4096) >= 4                                # the status word
    assert size(2048, 4088, 4096) == 0 and size(-1, 64, 64) == 0      # refused sizes


def test_wrappers_refuse_host_tensors_and_bad_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        block.add_rmsnorm_q8(x, torch.ones(64))
    with pytest.raises(TypeError, match="CUDA"):
        block.swiglu_q8(x)
    with pytest.raises(TypeError, match="CUDA"):
        block.quantize_q8(x)
    with pytest.raises(TypeError, match="int8"):
        block.dequantize_q8(x, torch.ones(4, 1))
    with pytest.raises(TypeError, match="CUDA"):
        block.route_scored(x, 2)
    with pytest.raises(TypeError, match="CUDA"):
        block.linear_q8(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4))


@pytest.mark.parametrize("kw", [
    dict(residual_out=P[2]),                                       # over the weights
    dict(residual_out=P[2], residual=None),
    dict(residual_out=P[0], ldx=8192),                             # x's rows are apart
    dict(residual_out=P[0], ldx=8192, residual=P[0], ldr=4096),    # x's and the residual's, one of them contiguous
    dict(residual_out=P[1], residual=P[1], x=P[1] + 2),            # in place for the residual, a shifted x
    dict(residual_out=P[0], weight=P[0]),                          # in place for x, which is the weights too
])
def test_norm_is_in_place_for_x_and_residual_only(lib, kw):
    assert _norm(lib, **kw) == INV
    assert "overlaps" in lib.wna16_moe_last_error().decode()


@pytest.mark.parametrize("over", ["xq", "xs", "wq", "ws", "bias"])
@pytest.mark.parametrize("in_place", [False, True])
def test_linear_is_in_place_for_the_addend_only(lib, over, in_place):
    kw = {over: P[5], "addend": P[5] if in_place else P[4]}
    assert _linear(lib, **kw) == INV
    assert "overlaps" in lib.wna16_moe_last_error().decode()


class _Rows:
    """What the argument checks look at of a CUDA tensor."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)

    def get_device(self):
        return 0

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P[0]


@pytest.mark.parametrize("bad,error", [((1 << 32), OverflowError), ((1 << 32) + 64, OverflowError), (-(1 << 40), OverflowError),
                                       (1 << 80, OverflowError), (64.0, TypeError), ("64", TypeError), (None, TypeError)])
def test_whole_numbers_are_not_cut_or_guessed(lib, bad, error):
    """An argument that is no whole number of 32 bits is refused as such, before anything is called
    (the entry point's address is 0 here)."""
    x, w = _Rows(torch.bfloat16, 4, 256), _Rows(torch.bfloat16, 256)
    q, s, s4 = _Rows(torch.int8, 4, 256), _Rows(torch.float32, 4, 1), _Rows(torch.float32, 4, 4)
    host = block._host
    for scales in (s, s4):
        with pytest.raises(error):
            host.quantize_q8(0, x, q, scales, bad, None)
        with pytest.raises(error):
            host.add_rmsnorm_q8(0, x, w, None, None, None, q, scales, 1e-6, bad, None)
        with pytest.raises(error):
            host.swiglu_q8(0, _Rows(torch.bfloat16, 4, 512), q, scales, 7.0, bad, None)
    ids, weights = _Rows(torch.int32, 4, 64), _Rows(torch.float32, 4, 64)
    good = [0, 8, 4, 0, 64, 1]
    for i in range(6):
        args = good[:i] + [bad] + good[i + 1:]
        with pytest.raises(error):
            host.route_scored(0, x, None, ids, weights, *args, 1.0, None)


@pytest.mark.parametrize("bad", ["7", None, [7.0]])
def test_numbers_are_numbers(lib, bad):
    x, w = _Rows(torch.bfloat16, 4, 256), _Rows(torch.bfloat16, 256)
    q, s = _Rows(torch.int8, 4, 256), _Rows(torch.float32, 4, 1)
    host = block._host
    for call in (lambda: host.add_rmsnorm_q8(0, x, w, None, None, None, q, s, bad, 0, None),
                 lambda: host.swiglu_q8(0, _Rows(torch.bfloat16, 4, 512), q, s, bad, 0, None),
                 lambda: host.route_scored(0, x, None, _Rows(torch.int32, 4, 8), _Rows(torch.float32, 4, 8), 0, 8, 4, 0, 8, 1, bad, None)):
        with pytest.raises(TypeError, match="float|number"):
            call()
