"""Host-side checks of the routed experts in 8-bit floats, without a GPU: every declared symbol is
exported, bad arguments are refused before any CUDA call (the pointers here are never dereferenced)."""
from __future__ import annotations

import os
import re

import pytest
import torch

from wna16_grouped_gemm_gb300 import binding, block, build, f8
from tests.test_block_host import _Rows

HEADER = os.path.join(os.path.dirname(binding.HEADER), "wna16_moe_f8.h")
P = [0x100000000000 * (i + 1) for i in range(10)]   # far apart
INV, UNS, SMALL = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED, binding.ERR_WORKSPACE_TOO_SMALL
BF, E4, FP, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    build.build()
    f8._load()
    return binding.load_library()


def test_every_declared_symbol_is_exported_by_both_builds(lib):
    with open(HEADER) as f:
        names = re.findall(r"WNA16_API\s+[\w\s\*]+?\b(wna16_\w+)\s*\(", f.read())
    assert len(names) == 6, names
    build.build(debug=True)
    for b in (lib, binding.load_debug_library()):
        for n in names:
            assert hasattr(b, n), n
    assert {"wna16_moe_" + n for n in f8._load()} == set(names)


def _sort(lib, *, x=P[0], ldx=4096, xs=P[1], groups=32, T=8, K=4096, type=3, ids=P[2], topk=8, E=256, begin=0, rows=P[3],
          rs=P[4], offsets=P[5], inv=P[6]):
    return lib.wna16_moe_sort_tokens(x, ldx, xs, groups, T, K, type, ids, topk, E, begin, rows, rs, offsets, inv, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=4), UNS), (dict(type=-1), UNS), (dict(T=-1), INV), (dict(K=0), INV), (dict(K=(1 << 26) + 1), UNS),
    (dict(T=1 << 31), UNS), (dict(T=1 << 29), UNS), (dict(topk=0), UNS), (dict(topk=1025), UNS), (dict(E=0), INV),
    (dict(E=1025), UNS), (dict(begin=-1), INV), (dict(begin=1 << 30), INV), (dict(ldx=4095), INV), (dict(ldx=1 << 41), INV),
    (dict(x=None, xs=None, rs=None), INV), (dict(rows=None), INV), (dict(xs=None), INV), (dict(rs=None), INV),
    (dict(x=None, rows=None), INV), (dict(groups=0), INV), (dict(groups=5000), INV), (dict(ids=None), INV),
    (dict(offsets=None), INV), (dict(inv=None), INV), (dict(ids=P[2] + 2), INV), (dict(x=P[0] + 1, type=0), INV),
    (dict(rows=P[3] + 2, type=2), INV), (dict(xs=P[1] + 1), INV), (dict(offsets=P[5] + 1), INV),
    (dict(rows=P[0] + 4096), INV), (dict(rows=P[2]), INV), (dict(rs=P[1]), INV), (dict(inv=P[2]), INV),
    (dict(offsets=P[6]), INV), (dict(rs=P[3] + 4096), INV),
])
def test_sort_refuses(lib, kw, code):
    assert _sort(lib, **kw) == code
    assert lib.wna16_moe_last_error().decode() != ""


def _unsort(lib, *, y=P[0], R=64, inv=P[1], w=P[2], addend=None, T=8, K=4096, topk=8, type=0, out=P[3]):
    return lib.wna16_moe_unsort_tokens(y, R, inv, w, addend, T, K, topk, type, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), UNS), (dict(T=-1), INV), (dict(K=0), INV), (dict(topk=0), UNS), (dict(topk=2000), UNS),
    (dict(T=1 << 29), UNS), (dict(R=-1), INV), (dict(R=1 << 31), INV), (dict(y=None), INV), (dict(inv=None), INV),
    (dict(out=None), INV), (dict(y=P[0] + 1), INV), (dict(inv=P[1] + 2), INV), (dict(w=P[2] + 2), INV),
    (dict(addend=P[4] + 1), INV), (dict(out=P[3] + 1), INV), (dict(out=P[0]), INV), (dict(out=P[2]), INV),
    (dict(addend=P[3] + 2), INV), (dict(out=P[1] - 4096), INV),
])
def test_unsort_refuses(lib, kw, code):
    assert _unsort(lib, **kw) == code
    assert lib.wna16_moe_last_error().decode() != ""


def _grad(lib, *, dout=P[0], inv=P[1], y=P[2], w=P[3], T=8, K=4096, topk=8, R=64, type=0, dy=P[4], dw=P[5]):
    return lib.wna16_moe_unsort_tokens_grad(dout, inv, y, w, T, K, topk, R, type, dy, dw, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), UNS), (dict(T=-1), INV), (dict(K=-1), INV), (dict(topk=0), UNS), (dict(R=-1), INV), (dict(dout=None), INV),
    (dict(inv=None), INV), (dict(y=None), INV), (dict(dw=None), INV), (dict(dy=None, y=None, dw=None), INV),
    (dict(dout=P[0] + 1), INV), (dict(y=P[2] + 1), INV), (dict(w=P[3] + 1), INV), (dict(dy=P[4] + 1), INV), (dict(dw=P[5] + 2), INV),
    (dict(dy=P[2]), INV), (dict(dy=P[0]), INV), (dict(dw=P[3]), INV), (dict(dw=P[4]), INV),
])
def test_unsort_grad_refuses(lib, kw, code):
    assert _grad(lib, **kw) == code
    assert lib.wna16_moe_last_error().decode() != ""


def _linear(lib, *, xq=P[0], xs=P[1], wq=P[2], ws=P[3], bias=None, addend=None, T=64, K=4096, N=4096, type=0, out=P[5],
            workspace=P[6], nbytes=256):
    return lib.wna16_moe_linear_f8(xq, xs, wq, ws, bias, addend, T, K, N, type, out, workspace, nbytes, None)


def _grouped(lib, *, xq=P[0], xs=P[1], wq=P[2], ws=P[3], offsets=P[4], E=8, T=64, K=4096, N=4096, type=0, out=P[5],
             workspace=P[6], nbytes=256):
    return lib.wna16_moe_grouped_linear_f8(xq, xs, wq, ws, offsets, E, T, K, N, type, out, workspace, nbytes, None)


@pytest.mark.parametrize("call", [_linear, _grouped])
@pytest.mark.parametrize("kw,code", [
    (dict(type=3), UNS), (dict(T=-1), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(K=4000), UNS), (dict(K=64), UNS),
    (dict(K=65536 + 128), UNS), (dict(T=1 << 30), UNS), (dict(N=1 << 24), UNS), (dict(xq=None), INV), (dict(wq=None), INV),
    (dict(xs=None), INV), (dict(ws=None), INV), (dict(xq=P[0] + 8), INV), (dict(wq=P[2] + 4), INV), (dict(xs=P[1] + 2), INV),
    (dict(ws=P[3] + 2), INV), (dict(out=None), INV), (dict(out=P[5] + 1), INV), (dict(workspace=P[6] + 2), INV),
    (dict(nbytes=3), SMALL), (dict(out=P[0] + 4096), INV), (dict(out=P[2]), INV), (dict(out=P[3]), INV),
    (dict(workspace=P[2]), INV), (dict(workspace=P[5] + 64), INV),
])
def test_linear_refuses(lib, call, kw, code):
    assert call(lib, **kw) == code
    assert lib.wna16_moe_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", [(dict(bias=P[4] + 1), INV), (dict(addend=P[4] + 1), INV), (dict(addend=P[5] + 2), INV), (dict(bias=P[5]), INV)])
def test_linear_refuses_bias_and_addend(lib, kw, code):
    assert _linear(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(offsets=None), INV), (dict(offsets=P[4] + 2), INV), (dict(E=0), INV), (dict(E=1025), UNS),
                                     (dict(E=1024, N=1 << 21), UNS), (dict(offsets=P[5]), INV)])
def test_grouped_refuses(lib, kw, code):
    assert _grouped(lib, **kw) == code


def _blocks(lib, *, w=P[0], E=2, N=300, K=512, se=300 * 512, sn=512, sk=1, type=0, q=P[1], scales=P[2]):
    return lib.wna16_moe_quantize_blocks_f8(w, E, N, K, se, sn, sk, type, q, scales, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), UNS), (dict(E=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=500), UNS), (dict(K=64), UNS),
    (dict(N=1 << 24), UNS), (dict(K=1 << 27), UNS), (dict(E=1 << 20, N=1 << 20, K=1 << 20), UNS), (dict(sn=511), INV),
    (dict(sk=2), INV), (dict(sn=1, sk=299), INV), (dict(sn=512, sk=0), INV), (dict(se=1000), INV), (dict(se=-1), INV),
    (dict(w=None), INV), (dict(q=None), INV), (dict(scales=None), INV), (dict(w=P[0] + 1), INV), (dict(scales=P[2] + 2), INV),
    (dict(q=P[0]), INV), (dict(scales=P[1]), INV),
])
def test_blocks_refuses(lib, kw, code):
    assert _blocks(lib, **kw) == code
    assert lib.wna16_moe_last_error().decode() != ""


def test_empty_batches_do_nothing(lib):
    assert _unsort(lib, T=0, y=None, inv=None, w=None, out=None) == 0
    assert _grad(lib, T=0, dout=None, inv=None, y=None, w=None, dy=None, dw=None) == 0
    assert _linear(lib, T=0, xq=None, xs=None, wq=None, ws=None, out=None, workspace=None, nbytes=0) == 0
    assert _grouped(lib, T=0, xq=None, xs=None, wq=None, ws=None, offsets=None, out=None, workspace=None, nbytes=0) == 0
    assert _blocks(lib, E=0, w=None, q=None, scales=None) == 0


class _More(_Rows):
    def __init__(self, dtype, *shape, device=0, contiguous=True):
        super().__init__(dtype, *shape)
        self.device_index, self.contiguous = device, contiguous

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return self.contiguous


def test_wrappers_refuse_other_shapes_types_and_devices(lib):
    """The checks before the entry point is called (its address is 0 here)."""
    h, T, K, k, E, N = block._host, 4, 256, 2, 8, 300
    ids, inv, off = _More(I32, T, k), _More(I32, T, k), _More(I32, E + 1)
    x, xs, rows, rs = _More(E4, T, K), _More(FP, T, 2), _More(E4, T * k, K), _More(FP, T * k, 2)

    def refused(error, name, *args):
        with pytest.raises(error):
            getattr(h, name)(0, *args, None)

    refused(TypeError, "sort_tokens", x, xs, _More(FP, T, k), E, 0, rows, rs, off, inv)
    refused(ValueError, "sort_tokens", _More(E4, T + 1, K), xs, ids, E, 0, rows, rs, off, inv)
    refused(TypeError, "sort_tokens", x, xs, ids, E, 0, _More(BF, T * k, K), rs, off, inv)
    refused(ValueError, "sort_tokens", x, xs, ids, E, 0, _More(E4, T, K), rs, off, inv)
    refused(ValueError, "sort_tokens", x, xs, ids, E + 1, 0, rows, rs, off, inv)
    refused(ValueError, "sort_tokens", x, xs, ids, E, 0, rows, rs, off, _More(I32, T, k + 1))
    refused(ValueError, "sort_tokens", x, xs, ids, E, 0, rows, rs, off, _More(I32, T, k, device=1))
    refused(ValueError, "sort_tokens", x, xs, _More(I32, T, k, contiguous=False), E, 0, rows, rs, off, inv)
    refused(OverflowError, "sort_tokens", x, xs, ids, 1 << 40, 0, rows, rs, off, inv)
    refused(TypeError, "sort_tokens", x, xs, ids, E, 0.5, rows, rs, off, inv)
    y, w, out = _More(BF, T * k, K), _More(FP, T, k), _More(BF, T, K)
    refused(TypeError, "unsort_tokens", rows, inv, w, None, out)
    refused(ValueError, "unsort_tokens", y, inv, _More(FP, T, k + 1), None, out)
    refused(ValueError, "unsort_tokens", y, inv, w, _More(BF, T + 1, K), out)
    refused(TypeError, "unsort_tokens", y, inv, w, _More(FP, T, K), out)
    refused(ValueError, "unsort_tokens", y, inv, w, None, _More(BF, T + 1, K))
    refused(ValueError, "unsort_tokens_grad", out, inv, _More(BF, T * k, K + 8), w, y, w)
    refused(ValueError, "unsort_tokens_grad", out, inv, y, w, _More(BF, T, K), w)
    refused(TypeError, "unsort_tokens_grad", out, inv, _More(FP, T * k, K), w, y, w)
    wq, ws = _More(E4, N, K), _More(FP, 3, 2)
    refused(ValueError, "linear_f8", x, _More(FP, T, 1), wq, ws, None, None, _More(BF, T, N), None)
    refused(ValueError, "linear_f8", x, xs, wq, _More(FP, N, 2), None, None, _More(BF, T, N), None)
    refused(ValueError, "linear_f8", x, xs, _More(E4, E, N, K), ws, None, None, _More(BF, T, N), None)
    refused(TypeError, "linear_f8", _More(torch.int8, T, K), xs, wq, ws, None, None, _More(BF, T, N), None)
    refused(ValueError, "linear_f8", x, xs, wq, ws, _More(FP, N + 1), None, _More(BF, T, N), None)
    w3, ws3 = _More(E4, E, N, K), _More(FP, E, 3, 2)
    refused(ValueError, "grouped_linear_f8", x, xs, wq, ws, off, _More(BF, T, N), None)
    refused(ValueError, "grouped_linear_f8", x, xs, w3, _More(FP, E, 2, 2), off, _More(BF, T, N), None)
    refused(ValueError, "grouped_linear_f8", x, xs, w3, ws3, _More(I32, E), _More(BF, T, N), None)
    refused(ValueError, "grouped_linear_f8", x, xs, w3, ws3, off, _More(BF, T, N + 1), None)
    refused(ValueError, "quantize_blocks_f8", _More(BF, N), _More(E4, N), _More(FP, 3))
    refused(ValueError, "quantize_blocks_f8", _More(BF, N, K), _More(E4, N, K), _More(FP, 2, 2))
    refused(ValueError, "quantize_blocks_f8", _More(BF, E, N, K), _More(E4, N, K), ws3)


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 256, dtype=BF)
    ids = torch.zeros(4, 2, dtype=I32)
    for call in (lambda: f8.sort_tokens(x, ids, 8), lambda: f8.unsort_tokens(x, ids), lambda: f8.unsort_tokens_grad(x, ids),
                 lambda: f8.linear_f8(x, x, x, x), lambda: f8.quantize_blocks_f8(x)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
