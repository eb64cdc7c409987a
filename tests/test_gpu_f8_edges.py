"""Routed experts in 8-bit floats on the GPU: what the documentation allows and the operators' first tests
(test_gpu_f8.py, whose tolerances and helpers these use) do not reach."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_f8 import BF, E4, FP, I32, check_sort, lists_ref, make_ids, moe  # noqa: F401  (moe: the fixture)
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
