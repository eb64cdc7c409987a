"""Routed experts in 8-bit floats on the GPU: what the documentation allows and the operators' first tests
(test_gpu_f8.py, whose tolerances and helpers these use) do not reach."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_f8 import (BF, E4, FP, I32, check_sort, lists_ref, make_ids, moe, product_ref,  # noqa: F401  (moe: the fixture)
                               product_tol, rows_f8)
from tests.test_gpu_block import U, check, half_step, randn

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


@pytest.mark.parametrize("R,mine,before", [
    (24, 11, (0, 1, 5, 8, 13)),                    # a mean of 4: tiles of 16 rows
    (60, 37, (0, 3, 16, 21, 23)),                  # of 10: 32 rows
    (200, 140, (0, 1, 31, 32, 47, 60)),            # of 33: 64 rows
    (600, 300, (0, 1, 33, 64, 127, 129, 300)),     # of 100: 128 rows
])
@pytest.mark.parametrize("K,N", [(1024, 300), (640, 264)])
@pytest.mark.parametrize("dt", [BF, FP])
def test_a_row_does_not_depend_on_its_neighbours(moe, R, mine, before, K, N, dt):  # noqa: F811
    """An expert's rows, moved to other places of the tiles among other experts' rows, some of them NaN in codes, scales and weights:
    the same bits (the numbers of rows and experts, which choose the kernel, stay).  And they are those of one weight's product."""
    E, e = 6, 3
    xq, xs = rows_f8(mine, K, 5)
    wq = rows_f8(E * N, K, 6)[0].view(E, N, K)
    ws = torch.exp(randn(E * -(-N // 128), K // 128, seed=7)).view(E, -1, K // 128) * 0.001
    bad_w = torch.full_like(wq.view(torch.uint8), 0x7f).view(E4)
    bad_w[e] = wq[e]
    first = None
    for at in before:
        for poison in (False, True):
            q, s = rows_f8(R, K, at)
            if poison:
                q = torch.full_like(q.view(torch.uint8), 0x7f).view(E4)
                s = torch.full_like(s, float("nan"))
            q[at:at + mine], s[at:at + mine] = xq, xs
            behind = R - at - mine
            counts = [at // 2, 0, at - at // 2, mine, behind // 3, behind - behind // 3]
            offsets = torch.tensor([0, *np.cumsum(counts)], dtype=I32, device="cuda")
            out = moe.grouped_linear_f8(q, s, bad_w if poison else wq, ws, offsets, dtype=dt)
            got = out[at:at + mine]
            assert bool(got.isfinite().all())
            others = torch.cat([out[:at], out[at + mine:]])
            assert bool(others.isnan().all() if poison else others.isfinite().all())
            first = got.clone() if first is None else first
            assert torch.equal(got, first), (at, poison)
    ref, S = product_ref(xq, xs, wq[e], ws[e])
    check(first, ref, half_step(dt) + U, "experts", extra=product_tol(K, S))
    h = half_step(dt) + U      # both are within h |ref| + tol of ref, and |ref| within (|other| + tol) / (1 - h)
    check(first, moe.linear_f8(xq, xs, wq[e], ws[e], dtype=dt).double(), 2 * h * (1 + 2 * h), "one weight", extra=2 * (1 + 2 * h) * product_tol(K, S))


def test_products_that_overlap_share_nothing(moe):  # noqa: F811
    """Products of several kernels and plans (two of them with a K shared over clusters, none with a workspace), queued on four
    streams from graphs, so that they run at the same time: each gives what it gives alone."""
    calls = [(64, 4096, 2048), (100, 8192, 256), (4, 4096, 4096), (700, 2048, 1024), (30, 16384, 128), (300, 1024, 520)]
    streams, graphs, inputs = [torch.cuda.Stream() for _ in range(4)], [], []
    for i, s in enumerate(streams):
        mine = []
        for T, K, N in calls[i:] + calls[:i]:
            xq, xs = rows_f8(T, K, T)
            wq, ws = rows_f8(N, K, T + 1)[0], torch.exp(randn(-(-N // 128), K // 128, seed=T + 2)) * 0.001
            mine.append((xq, xs, wq, ws, torch.zeros(T, N, device="cuda"), moe.linear_f8(xq, xs, wq, ws, dtype=FP)))
        inputs.append(mine)
    torch.cuda.synchronize()
    for s, mine in zip(streams, inputs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(4):
                for xq, xs, wq, ws, out, _ in mine:
                    moe.linear_f8(xq, xs, wq, ws, out=out)
        graphs.append(g)
    for _ in range(8):
        for mine in inputs:
            for c in mine:
                c[4].fill_(-1.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for mine in inputs:
            for c in mine:
                assert torch.equal(c[4], c[5]), tuple(c[0].shape)
