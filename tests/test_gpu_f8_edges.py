"""Routed experts in 8-bit floats on the GPU: what the documentation allows and the operators' first tests
(test_gpu_f8.py, whose tolerances and helpers these use) do not reach."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_f8 import BF, E4, FP, I32, check_sort, lists_ref, make_ids, moe, rows_f8  # noqa: F401  (moe: the fixture)
from tests.test_gpu_block import randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,topk,total", [(769, 8, 256), (6145, 1, 1024), (6146, 1, 3), (1700, 8, 512)])
def test_lists_of_a_cluster_are_the_same_every_time(moe, T, topk, total):  # noqa: F811
    """Lists of many slots are made by a cluster of blocks, of which the last have few slots or none here and are at the
    exchange of the counts first.  Replayed many times beside another stream's copies, every list is the right one."""
    ids = make_ids(T, topk, total, seed=T, skew=True, padding=0.1)
    _, inv_ref, off_ref = lists_ref(ids, total, 0)
    runs = 20
    offs = [torch.full((total + 1,), -7, dtype=I32, device="cuda") for _ in range(runs)]
    invs = [torch.full((T, topk), -7, dtype=I32, device="cuda") for _ in range(runs)]
    moe.sort_tokens(None, ids, total)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o, i in zip(offs, invs):
            moe.sort_tokens(None, ids, total, offsets=o, inv=i)
    side = torch.cuda.Stream()
    a, b = torch.zeros(1 << 24, device="cuda"), torch.zeros(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            b.copy_(a)
        graph.replay()
    torch.cuda.synchronize()
    for o, i in zip(offs, invs):
        assert np.array_equal(o.cpu().numpy(), off_ref) and np.array_equal(i.cpu().numpy(), inv_ref)


def test_gradient_of_no_rows(moe):  # noqa: F811
    """A share of the experts that got no slot, with buffers of no rows."""
    inv = torch.full((5, 3), -1, dtype=I32, device="cuda")
    d, none = randn(5, 64, dtype=BF), torch.empty(0, 64, dtype=BF, device="cuda")
    dy, dw = moe.unsort_tokens_grad(d, inv, dy=none)
    assert dy is none and dw is None
    dy, dw = moe.unsort_tokens_grad(d, inv, none, torch.rand(5, 3, device="cuda"), dy=torch.empty_like(none))
    assert dy.shape == (0, 64) and torch.equal(dw, torch.zeros(5, 3, device="cuda"))
    assert torch.equal(moe.unsort_tokens(none, inv), torch.zeros_like(d))


@pytest.fixture
def checked(moe):  # noqa: F811
    """The entry points of the bounds-checked build in the place of the release build's; gives the word of its index checks."""
    import ctypes

    from wna16_grouped_gemm_gb300 import binding, build, f8
    build.build(debug=True)
    debug, saved = binding.load_debug_library(), f8._load()
    entries = f8.declare(debug)

    def status():
        word = ctypes.c_int(99)
        assert debug.wna16_moe_debug_index_status(ctypes.byref(word)) == 0
        return word.value

    def use(on):
        f8._entries = entries if on else saved

    use(True)
    yield status, use
    use(False)


@pytest.mark.parametrize("T,topk,total,E,begin,K,dt", [
    (3, 2, 8, 8, 0, 17, BF), (700, 8, 64, 64, 0, 264, E4), (769, 8, 256, 64, 64, 130, BF), (9363, 7, 64, 64, 0, 16, FP), (2, 1000, 6, 6, 0, 100, BF),
    (20000, 5, 1024, 1024, 0, 20, BF), (1, 1, 1, 1, 0, 1, E4),
])
def test_bounds_checked_rows(moe, checked, T, topk, total, E, begin, K, dt):  # noqa: F811
    """Lists, rows and the way back: the index checks find nothing, and the bits are the release build's."""
    status, use = checked
    ids = make_ids(T, topk, total, seed=T, skew=True, padding=0.2)
    x = randn(T, K, seed=T, scale=30.0).to(dt)
    outs = []
    for on in (True, False):
        use(on)
        rows, _, _, inv = check_sort(moe, x, ids, E, begin)
        if dt != E4:
            y, d, w = randn(T * topk, K, seed=2, dtype=dt), randn(T, K, seed=3, dtype=dt), torch.rand(T, topk, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
            dy, dw = moe.unsort_tokens_grad(d, inv, y, w, dy=torch.zeros_like(y))
            outs.append([rows, moe.unsort_tokens(y, inv, w), dy, dw])
        else:
            outs.append([rows])
    assert status() == 0
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("counts,K,N,dt", [
    ([4], 256, 17, BF), ([40], 4096, 130, FP), ([77], 8192, 640, BF), ([200], 512, 264, FP), ([700], 1024, 513, BF), ([1000], 128, 1, FP),
    ([1, 0, 2, 5, 0, 0, 1], 2048, 1000, BF), ([9] * 30, 384, 264, FP), ([20, 40, 0, 33, 65], 640, 129, BF), ([300, 2, 0, 41, 127, 128, 129], 1024, 520, FP),
    ([0, 0, 0], 128, 64, BF),
])
def test_bounds_checked_products(moe, checked, counts, K, N, dt):  # noqa: F811
    """Products with one weight and with several: the status word stays at OK, and the bits are the release build's."""
    status, use = checked
    R, E = sum(counts), len(counts)
    xq, xs = rows_f8(max(R, 1), K, 1)
    wq = rows_f8(E * N, K, 2)[0].view(E, N, K)
    ws = torch.exp(randn(E * -(-N // 128), K // 128, seed=3)).view(E, -1, K // 128) * 0.001
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=I32, device="cuda")
    outs = []
    for on in (True, False):
        use(on)
        work = torch.full((256,), 77, dtype=torch.uint8, device="cuda")
        out = torch.zeros(xq.shape[0], N, dtype=dt, device="cuda")
        if E == 1:
            moe.linear_f8(xq, xs, wq[0], ws[0], out=out, workspace=work)
        else:
            moe.grouped_linear_f8(xq, xs, wq, ws, offsets, out=out, workspace=work)
        assert moe.read_status(work) == moe.OK
        outs.append(out)
    assert status() == 0 and torch.equal(*outs)
