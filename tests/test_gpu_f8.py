"""Routed experts in 8-bit floats on the GPU, against plain 64-bit computations of their definitions.

Tolerances, with u = 2^-24 (fp32 half step) and e = eps(type) / 2 (the output's half step):
  sort    copies: equal bit for bit.
  unsort  a chain of topk fused multiply-adds and the addend: (topk + 2) u of the magnitudes added; then e.
  grad    dy: one product (u), then e.  dweights: at most K / 256 + 64 serial additions of fused products:
          that many u of the magnitudes added.
  linear  a block's sum: exact products; each tensor core instruction adds 32 of them to a sum with every term
          cut at no more than 2^-25 of the largest magnitude and the result at 2^-23: 4 (32 * 2^-25 + 2^-23) =
          4.5 * 2^-20 of the block's magnitudes; the scales' product, and a fused multiply-add per block and
          at most 8 parts: (blocks + 10) u; bias, addend: 2 u; then e.  All of S = sum |x w| and the addends.
  blocks  m / 448: u of the scale.  A code is off by half a step, 2^-4 of the value or 2^-10 of the scale (below
          2^-6, steps are 2^-9), the quotient and the product before it by 2 u of the value, the scale by u.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_block import U, check, half_step, randn

pytestmark = pytest.mark.gpu

BF, HF, FP, E4, I8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int8, torch.int32
B = 128


@pytest.fixture(scope="module")
def moe():
    import wna16_grouped_gemm_gb300 as m
    from wna16_grouped_gemm_gb300 import build
    build.build()
    m.load_library()
    return m


def floor_of(dt):
    """Half the smallest step: fp16 has subnormal numbers in reach."""
    return 2.0 ** -25 if dt == HF else 0.0


# ---------------------------------------------------------------- sort and unsort


def make_ids(T, topk, total, seed=0, skew=False, padding=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.rand(T, total, generator=g, device="cuda")
    if skew:
        z = z - 0.9 * (torch.arange(total, device="cuda") / total)
    ids = z.argsort(dim=1, descending=True)[:, :topk] if topk <= total else torch.randint(total, (T, topk), generator=g, device="cuda")
    pad = torch.rand(T, ids.shape[1], generator=g, device="cuda") < padding
    return torch.where(pad, -1, ids).to(I32).contiguous()


def lists_ref(ids, E, begin):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64) - begin
    kept = np.flatnonzero((flat >= 0) & (flat < E))
    order = kept[np.argsort(flat[kept], kind="stable")]
    inv = np.full(flat.size, -1)
    inv[order] = np.arange(order.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=E))])
    return order, inv.reshape(ids.shape), offsets


def check_sort(moe, x, ids, E, begin=0, scales=None, **kw):
    T, topk = ids.shape
    order, inv_ref, off_ref = lists_ref(ids, E, begin)
    fill = torch.full((T * topk, x.shape[1]), 7, device="cuda").to(x.dtype)
    srows = None if scales is None else torch.full((T * topk, scales.shape[1]), 7.0, device="cuda")
    rows, rs, off, inv = moe.sort_tokens(x, ids, E, scales=scales, expert_begin=begin, rows=fill.clone(), row_scales=srows, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(inv.cpu().numpy(), inv_ref)
    assert np.array_equal(off.cpu().numpy(), off_ref)
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    token = torch.from_numpy(order // topk).cuda()
    n = token.numel()
    assert torch.equal(bits(rows[:n]), bits(x[token]))
    assert torch.equal(bits(rows[n:]), bits(fill[n:])), "rows behind the last expert"
    if scales is not None:
        assert torch.equal(rs[:n], scales[token]) and bool((rs[n:] == 7).all())
    return rows, rs, off, inv


SORTS = [
    # T, topk, total, E, begin, K, type, skew, padding
    (1, 1, 1, 1, 0, 16, BF, False, 0.0), (1, 8, 256, 256, 0, 4096, E4, False, 0.0), (4, 8, 256, 256, 0, 4096, E4, False, 0.0),
    (3, 2, 8, 8, 0, 1, I8, False, 0.0), (5, 3, 16, 16, 0, 1021, E4, False, 0.0), (7, 4, 32, 8, 8, 130, BF, False, 0.0),
    (9, 2, 64, 64, 0, 515, FP, True, 0.3), (33, 6, 160, 40, 120, 2048, HF, True, 0.0), (2, 1, 1024, 1024, 0, 256, BF, False, 0.0),
    (100, 40, 64, 64, 0, 128, BF, False, 0.1), (513, 8, 256, 256, 0, 256, E4, False, 0.0), (512, 8, 256, 128, 128, 136, BF, True, 0.0),
    (600, 7, 1024, 1024, 0, 100, HF, False, 0.2), (2047, 8, 256, 64, 64, 384, FP, True, 0.0), (5000, 1, 8, 8, 0, 17, I8, True, 0.0),
    (8192, 8, 256, 256, 0, 512, BF, True, 0.0), (300, 33, 3, 3, 0, 64, BF, False, 0.0), (3, 1024, 5, 5, 0, 32, E4, False, 0.5),
    (70, 100, 9, 9, 0, 48, HF, False, 0.0), (40000, 8, 60, 60, 0, 32, E4, False, 0.0),
    # around the largest batch that is counted by its own blocks, and lists of every size by the cluster
    (768, 8, 256, 256, 0, 128, BF, False, 0.0), (769, 8, 256, 256, 0, 128, BF, True, 0.3), (6145, 1, 1024, 1024, 0, 64, HF, False, 0.0),
    (3000, 7, 1024, 512, 512, 72, FP, True, 0.1), (9363, 7, 64, 64, 0, 16, E4, True, 0.0), (20000, 5, 1024, 1024, 0, 20, BF, True, 0.0),
    (2, 800, 6, 6, 0, 1000, BF, True, 0.0), (7000, 1, 1, 1, 0, 33, I8, False, 0.5),
]


@pytest.mark.parametrize("T,topk,total,E,begin,K,dt,skew,padding", SORTS)
def test_sort(moe, T, topk, total, E, begin, K, dt, skew, padding):
    x = randn(T, K, seed=T, scale=30.0).to(dt)
    ids = make_ids(T, topk, total, seed=T + topk, skew=skew, padding=padding)
    scales = randn(T, max(1, K // B), seed=5) if dt in (E4, I8) else None
    check_sort(moe, x, ids, E, begin, scales)
    r = moe.sort_tokens(None, ids, E, expert_begin=begin)
    order, inv, off = lists_ref(ids, E, begin)
    assert r[0] is None and r[1] is None and np.array_equal(r[2].cpu(), off) and np.array_equal(r[3].cpu(), inv)


@pytest.mark.parametrize("T", [6, 900])
def test_sort_no_slot_stays(moe, T):
    x = randn(T, 64, dtype=BF)
    for value in (-1, 8, 2 ** 31 - 1, -2 ** 31):
        ids = torch.full((T, 8), value, dtype=I32, device="cuda")
        check_sort(moe, x, ids, 8)
        check_sort(moe, x, ids, 8, begin=2 ** 30 - 1)
    check_sort(moe, x, torch.full((T, 8), 3, dtype=I32, device="cuda"), 8)    # one expert has every slot


def test_sort_empty(moe):
    rows, rs, off, inv = moe.sort_tokens(randn(0, 64, dtype=BF), torch.empty(0, 4, dtype=I32, device="cuda"), 16,
                                         offsets=torch.full((17,), 9, dtype=I32, device="cuda"))
    assert rows.shape == (0, 64) and inv.shape == (0, 4) and bool((off == 0).all())


@pytest.mark.parametrize("T", [37, 1500])
def test_sort_strided_and_unaligned(moe, T):
    ids = make_ids(T, 4, 32, seed=3)
    for dt in (BF, E4, FP):
        for off, K, width in ((0, 256, 272), (8, 250, 266), (1, 255, 257), (3, 64, 80)):
            check_sort(moe, randn(T, width, seed=off, scale=30.0).to(dt)[:, off:off + K], ids, 32)


def ref_unsort(y, inv, w, add=None):
    """(64-bit result, magnitudes added)"""
    T, topk = inv.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for j in range(topk):
        i = inv[:, j].long()
        used = ((i >= 0) & (i < y.shape[0])).unsqueeze(1)
        v = torch.where(used, y.double()[i.clamp(0, y.shape[0] - 1)], 0.0) * (1.0 if w is None else torch.where(used, w.double()[:, j:j + 1], 0.0))
        out += v
        mag += v.abs()
    if add is not None:
        out += add.double()
        mag += add.double().abs()
    return out, mag


UNSORTS = [
    # T, topk, E, K, type, weights, addend, padding
    (1, 1, 4, 8, BF, True, False, 0.0), (4, 8, 256, 4096, BF, True, False, 0.0), (5, 3, 8, 1021, BF, True, True, 0.3),
    (7, 8, 16, 2056, HF, False, False, 0.2), (33, 6, 64, 4097, FP, True, True, 0.0), (3, 20, 40, 640, BF, True, False, 0.0),
    (300, 8, 256, 5120, BF, True, True, 0.1), (2047, 8, 64, 512, FP, False, False, 0.5), (6, 9, 12, 3, HF, True, False, 0.0),
    (4000, 2, 8, 2048, BF, True, False, 0.0),
]


@pytest.mark.parametrize("T,topk,E,K,dt,weighted,added,padding", UNSORTS)
def test_unsort(moe, T, topk, E, K, dt, weighted, added, padding):
    ids = make_ids(T, topk, E, seed=K, padding=padding)
    inv = moe.sort_tokens(None, ids, E)[3]
    y = randn(T * topk, K, seed=1, dtype=dt)
    y[int((inv >= 0).sum()):] = float("nan")                     # rows that no slot has are not read
    w = torch.rand(T, topk, device="cuda") if weighted else None
    add = randn(T, K, seed=2, dtype=dt) if added else None
    out = moe.unsort_tokens(y, inv, w, addend=add)
    ref, mag = ref_unsort(y, inv, w, add)
    check(out, ref, half_step(dt) + U, "unsort", floor=floor_of(dt), extra=(topk + 2) * U * mag)
    if added:
        buf = add.clone()
        assert moe.unsort_tokens(y, inv, w, addend=buf, out=buf) is buf and torch.equal(buf, out)


@pytest.mark.parametrize("T,topk,E,K,dt,weighted,added,padding", UNSORTS)
def test_unsort_grad(moe, T, topk, E, K, dt, weighted, added, padding):
    ids = make_ids(T, topk, E, seed=K, padding=padding)
    inv = moe.sort_tokens(None, ids, E)[3]
    used = inv >= 0
    n = int(used.sum())
    y, d = randn(T * topk, K, seed=1, dtype=dt), randn(T, K, seed=2, dtype=dt)
    y[n:] = float("nan")
    w = torch.rand(T, topk, device="cuda") if weighted else None
    fill = torch.full_like(y, 5.0)
    dy, dw = moe.unsort_tokens_grad(d, inv, y, w, dy=fill)
    assert bool((dy[n:] == 5.0).all())
    t = torch.arange(T, device="cuda").unsqueeze(1).expand(T, topk)[used]
    at = inv[used].long()
    ref = d.double()[t] * (1.0 if w is None else w.double()[used].unsqueeze(1))
    check(dy[at], ref, half_step(dt) + 2 * U, "dy", floor=floor_of(dt))
    rows = y.double()[at] * d.double()[t]
    assert bool((dw[~used] == 0).all())
    check(dw[used], rows.sum(dim=1), 0.0, "dweights", extra=(K / 256 + 64) * U * rows.abs().sum(dim=1))
    # each alone
    only = moe.unsort_tokens_grad(d, inv, y, w, want_dy=False)
    assert only[0] is None and torch.equal(only[1], dw)
    only = moe.unsort_tokens_grad(d, inv, None, w, dy=torch.full_like(y, 5.0))
    assert only[1] is None and torch.equal(only[0], dy)


@pytest.mark.parametrize("T,topk,E,K,dt,weighted,added,padding", [
    # few slots per token: several runs of a row at a time, the last ones partly or wholly past its end
    (3000, 1, 16, 4096, BF, True, False, 0.0), (2500, 2, 8, 2568, FP, True, True, 0.2), (3000, 4, 64, 1544, HF, False, True, 0.1),
    (700, 2, 8, 16384, FP, True, False, 0.0), (1000, 4, 8, 4104, BF, True, True, 0.4), (4000, 1, 8, 8, FP, True, False, 0.5),
    (1, 2, 8, 8192, BF, True, True, 0.0), (1500, 3, 8, 3080, BF, False, False, 0.0), (1200, 2, 8, 1026, HF, True, False, 0.0),
])
def test_unsort_few_slots(moe, T, topk, E, K, dt, weighted, added, padding):
    test_unsort(moe, T, topk, E, K, dt, weighted, added, padding)
    test_unsort_grad(moe, T, topk, E, K, dt, weighted, added, padding)


def test_rows_past_32_bits(moe):
    """Elements and bytes past 2^31 and 2^32: the rows of the last experts and tokens."""
    T, topk, E, K = 9000, 8, 16, 32768
    x = torch.empty(T, K, dtype=HF, device="cuda")
    for a in range(0, T, 3000):
        x[a:a + 3000] = randn(3000, K, seed=a, dtype=HF)
    ids = make_ids(T, topk, E, seed=1)
    rows, _, off, inv = moe.sort_tokens(x, ids, E)
    order, inv_ref, off_ref = lists_ref(ids, E, 0)
    assert np.array_equal(inv.cpu().numpy(), inv_ref) and np.array_equal(off.cpu().numpy(), off_ref)
    for a in (0, T * topk // 2, T * topk - 500):
        assert torch.equal(rows[a:a + 500], x[torch.from_numpy(order[a:a + 500] // topk).cuda()])
    w = torch.rand(T, topk, device="cuda")
    out = moe.unsort_tokens(rows, inv, w)
    for t in (0, T // 2, T - 1):
        ref = (x[t].double() * w[t].double().sum())
        check(out[t], ref, half_step(HF) + 20 * U, "unsort", floor=floor_of(HF))
    dy, dw = moe.unsort_tokens_grad(x, inv, rows, w, dy=torch.empty_like(rows))
    for t in (0, T - 1):
        check(dy[inv[t].long()], x[t].double() * w[t].double().unsqueeze(1), half_step(HF) + 2 * U, "dy", floor=floor_of(HF))
        sq = (x[t].double() ** 2).sum()
        check(dw[t], sq.expand(topk), (K / 256 + 64) * U, "dweights")


def test_unsort_leaves_out_rows_outside(moe):
    """An inv outside [0, R) is not read."""
    y = randn(6, 128, dtype=BF)
    inv = torch.tensor([[0, 6], [-1, 5], [-7, 2 ** 31 - 1]], dtype=I32, device="cuda")
    out = moe.unsort_tokens(y, inv)
    assert torch.equal(out, torch.stack([y[0], y[5], torch.zeros_like(y[0])]))
    dy, dw = moe.unsort_tokens_grad(randn(3, 128, seed=4, dtype=BF), inv, y)
    assert bool((dw[[0, 1, 2, 2], [1, 0, 0, 1]] == 0).all()) and bool((dw[[0, 1], [0, 1]] != 0).all())
    assert torch.equal(moe.unsort_tokens(y[:0], inv), torch.zeros(3, 128, dtype=BF, device="cuda"))


def test_sort_and_unsort_keep_infinities_and_nan(moe):
    x = randn(4, 256, dtype=BF)
    x[0, 3], x[1, 4], x[2, 5] = float("inf"), float("-inf"), float("nan")
    ids = make_ids(4, 2, 8)
    rows, _, _, inv = check_sort(moe, x, ids, 8)
    out = moe.unsort_tokens(rows, inv, torch.full((4, 2), 0.5, device="cuda"))
    assert torch.equal(out.nan_to_num(9.0), x.nan_to_num(9.0)) and bool(out[2, 5].isnan())


def test_gradients_are_those_of_differences(moe):
    """With a loss of <dout, unsort(sort(x) * 1, weights)>, in fp32: central differences.  The loss is linear in
    x and in the weights, so a difference of step h is off by the sums' rounding only: 2 (topk + 2) u of the
    output's magnitudes per element, summed against |dout|, over 2 h."""
    T, topk, E, K, h = 6, 3, 5, 40, 0.5
    ids = make_ids(T, topk, E, seed=2, padding=0.2)
    x, d, w = randn(T, K, seed=1), randn(T, K, seed=2), torch.rand(T, topk, device="cuda")

    def loss(x, w):
        rows, _, _, inv = moe.sort_tokens(x, ids, E)
        out = moe.unsort_tokens(rows, inv, w)
        return float((out.double() * d.double()).sum()), rows, inv

    _, rows, inv = loss(x, w)
    dy, dw = moe.unsort_tokens_grad(d, inv, rows, w)
    dx = moe.unsort_tokens(dy, inv)
    _, mag = ref_unsort(rows.abs() + h, inv, w + h)
    tol = float((d.double().abs() * mag).sum()) * 2 * (topk + 2) * U / (2 * h)
    g = np.random.default_rng(0)
    for _ in range(20):
        t, k, j = int(g.integers(T)), int(g.integers(K)), int(g.integers(topk))
        up, down = x.clone(), x.clone()
        up[t, k] += h
        down[t, k] -= h
        got = (loss(up, w)[0] - loss(down, w)[0]) / float(up[t, k].double() - down[t, k].double())
        assert abs(got - float(dx[t, k])) <= tol + 8 * U * abs(got)
        up, down = w.clone(), w.clone()
        up[t, j] += h
        down[t, j] -= h
        got = (loss(x, up)[0] - loss(x, down)[0]) / float(up[t, j].double() - down[t, j].double())
        assert abs(got - float(dw[t, j])) <= tol + 64 * U * float((d[t].double() * x[t].double()).abs().sum())


# ---------------------------------------------------------------- products


def rows_f8(T, K, seed):
    q = randn(T, K, seed=seed, scale=120.0).clamp(-448, 448).to(E4)
    s = torch.exp(randn(T, K // B, seed=seed + 1)) * 0.01
    return q, s


def values(q, s):
    return q.double() * s.double().repeat_interleave(B, dim=1)


def block_values(q, s):
    return values(q, s.repeat_interleave(B, dim=0)[:q.shape[0]])


def product_ref(xq, xs, wq, ws):
    """(64-bit product, product of the magnitudes)"""
    x, w = values(xq, xs), block_values(wq, ws)
    return x @ w.t(), x.abs() @ w.abs().t()


def product_tol(K, S):
    return (4.5 * 2.0 ** -20 + (K // B + 12) * U) * S


def check_linear(moe, T, K, N, dt=BF, bias=False, add=False, seed=0, **kw):
    xq, xs = rows_f8(T, K, seed)
    wq, _ = rows_f8(N, K, seed + 10)
    ws = torch.exp(randn(-(-N // B), K // B, seed=seed + 12)) * 0.001
    b = randn(N, seed=seed + 13) if bias else None
    a = randn(T, N, seed=seed + 14, dtype=dt) if add else None
    out = moe.linear_f8(xq, xs, wq, ws, bias=b, addend=a, dtype=dt, **kw)
    ref, S = product_ref(xq, xs, wq, ws)
    extra = product_tol(K, S)
    for v in (b, a):
        if v is not None:
            ref, extra = ref + v.double(), extra + 3 * U * v.double().abs()
    check(out, ref, half_step(dt) + U, "linear", floor=floor_of(dt), extra=extra)
    return out


LINEARS = [(1, 128, 1), (1, 4096, 4096), (2, 256, 17), (4, 4096, 4096), (5, 384, 130), (8, 128, 256), (9, 2048, 1000), (16, 640, 128),
           (17, 1024, 264), (32, 4096, 512), (33, 128, 129), (64, 2048, 384), (77, 2048, 1000), (100, 896, 2000), (127, 256, 4096),
           (128, 512, 256), (129, 384, 257), (200, 4096, 1024), (256, 128, 128), (300, 1024, 513), (512, 2048, 2048), (1000, 256, 4104),
           (1, 65536, 40), (40, 32768, 96), (2500, 512, 300), (2048, 4096, 1536), (700, 8192, 640)]


@pytest.mark.parametrize("T,K,N", LINEARS)
@pytest.mark.parametrize("dt", [BF, HF, FP])
def test_linear(moe, T, K, N, dt):
    check_linear(moe, T, K, N, dt, seed=T + N)


@pytest.mark.parametrize("T,K,N", [(3, 256, 130), (40, 1024, 250), (150, 512, 96), (600, 2048, 520)])
@pytest.mark.parametrize("dt", [BF, FP])
def test_linear_bias_and_addend(moe, T, K, N, dt):
    plain = check_linear(moe, T, K, N, dt, seed=5)
    assert not torch.equal(plain, check_linear(moe, T, K, N, dt, bias=True, seed=5))
    check_linear(moe, T, K, N, dt, add=True, seed=5)
    check_linear(moe, T, K, N, dt, bias=True, add=True, seed=5)
    buf = randn(T, N, seed=19, dtype=dt)
    xq, xs = rows_f8(T, K, 5)
    wq, ws = rows_f8(N, K, 15)[0], torch.exp(randn(-(-N // B), K // B, seed=17)) * 0.001
    first = moe.linear_f8(xq, xs, wq, ws, addend=buf)
    assert first.dtype == dt and moe.linear_f8(xq, xs, wq, ws, addend=buf, out=buf) is buf and torch.equal(first, buf)


@pytest.mark.parametrize("T", [4, 70, 400])
def test_linear_extreme_codes_and_scales(moe, T):
    """Largest and smallest codes, zero scales, scales far apart."""
    K, N = 1024, 384
    wq, ws = rows_f8(N, K, 3)[0], torch.full((3, K // B), 0.5, device="cuda")
    xq, xs = rows_f8(T, K, 7)
    xq[0] = 448.0
    wq[0] = -448.0
    wq[1] = 2.0 ** -9
    xq[1] = 2.0 ** -9
    xs[2] = 0.0
    xs[3] = 2.0 ** -60
    ws[1, 3], ws[2, 0], ws[2, 1] = 0.0, 2.0 ** 40, 2.0 ** -40
    out = moe.linear_f8(xq, xs, wq, ws, dtype=FP)
    ref, S = product_ref(xq, xs, wq, ws)
    check(out, ref, U, "linear", extra=product_tol(K, S))
    assert bool((out[2] == 0).all())
    xs[0, 1], xs[1, 2] = float("nan"), float("inf")      # rows that were not finite: codes 0
    xq[0, B:2 * B], xq[1, 2 * B:3 * B] = 0.0, 0.0
    out = moe.linear_f8(xq, xs, wq, ws, dtype=FP)
    assert bool(out[:2].isnan().all()) and bool(out[2:].isfinite().all())


@pytest.mark.parametrize("T", [2, 40, 300])
def test_linear_codes_that_are_nan(moe, T):
    """A NaN code makes its row or its channel NaN, and no other."""
    K, N = 512, 264
    xq, xs = rows_f8(T, K, 1)
    wq, ws = rows_f8(N, K, 2)[0], torch.full((3, K // B), 0.001, device="cuda")
    xq.view(torch.uint8)[1, 200] = 0x7f
    wq.view(torch.uint8)[N - 1, 500] = 0xff
    bad = moe.linear_f8(xq, xs, wq, ws, dtype=FP).isnan()
    want = torch.zeros_like(bad)
    want[1], want[:, N - 1] = True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T", [3, 50, 300])
def test_linear_is_reproducible(moe, T):
    a = check_linear(moe, T, 2048, 520, FP, seed=1)
    for _ in range(3):
        assert torch.equal(a, check_linear(moe, T, 2048, 520, FP, seed=1))


@pytest.mark.parametrize("T", [2, 60, 500])
def test_linear_unaligned_output(moe, T):
    """Outputs, biases and addends need the alignment of their elements only, as do scales."""
    K, N = 512, 200
    xq, xs = rows_f8(T, K, 1)
    wq, ws = rows_f8(N, K, 2)[0], torch.exp(randn(2, K // B, seed=3)) * 0.001
    a = moe.linear_f8(xq, xs, wq, ws)
    buf = torch.zeros(T * N + 9, dtype=BF, device="cuda")
    out = buf[1:1 + T * N].view(T, N)
    sb = torch.zeros(T * 4 + 1, device="cuda")
    sb[1:] = xs.reshape(-1)
    wb = torch.zeros(9, device="cuda")
    wb[1:] = ws.reshape(-1)
    moe.linear_f8(xq, sb[1:].view(T, 4), wq, wb[1:].view(2, 4), out=out)
    assert torch.equal(out, a) and float(buf[0]) == 0 and bool((buf[1 + T * N:] == 0).all())


def test_linear_status(moe):
    ws = torch.full((16,), 0x5a, dtype=torch.uint8, device="cuda")
    for T in (3, 60, 300):
        check_linear(moe, T, 1024, 300, workspace=ws[:4], seed=1)
        assert moe.read_status(ws) == moe.OK
        ws.fill_(0x5a)
    with pytest.raises(moe.Wna16Error):
        check_linear(moe, 3, 1024, 300, workspace=ws[:3], seed=1)
    assert bool((ws == 0x5a).all())


def check_grouped(moe, counts, K, N, dt=BF, first=0, behind=0, seed=0, **kw):
    E = len(counts)
    offsets = torch.tensor([first, *(first + np.cumsum(counts))], dtype=I32, device="cuda")
    n = int(offsets[-1])
    R = n + behind
    xq, xs = rows_f8(R, K, seed)
    xs[n:] = float("nan")                                       # rows of no expert
    xs[:first] = float("nan")
    wq = rows_f8(E * N, K, seed + 3)[0].view(E, N, K)
    ws = torch.exp(randn(E, -(-N // B), K // B, seed=seed + 6)) * 0.001
    out = torch.full((R, N), 3.0, dtype=dt, device="cuda")
    moe.grouped_linear_f8(xq, xs, wq, ws, offsets, out=out, **kw)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        ref, S = product_ref(xq[a:b], xs[a:b], wq[e], ws[e])
        check(out[a:b], ref, half_step(dt) + U, f"expert {e}", floor=floor_of(dt), extra=product_tol(K, S))
    assert bool((out[:first] == 3).all()) and bool((out[n:] == 3).all())
    return out


GROUPED = [
    # rows per expert, K, N, first row, rows behind
    ([1], 128, 1, 0, 0), ([0, 3, 0, 1], 256, 130, 0, 2), ([2] * 16, 4096, 512, 0, 0), ([1, 0, 2, 5, 0, 0, 1], 2048, 1000, 3, 4),
    ([17, 16, 15, 1, 33], 512, 264, 0, 1), ([64, 1, 0, 65, 130], 640, 384, 5, 0), ([0] * 7, 256, 128, 0, 4), ([300, 2, 0, 41, 127, 128, 129], 1024, 520, 1, 7),
    ([256] * 4, 512, 256, 0, 0), ([1000, 3], 384, 300, 0, 0), ([5] * 200, 256, 200, 0, 3), ([0, 0, 700], 2048, 1024, 0, 0),
]


@pytest.mark.parametrize("counts,K,N,first,behind", GROUPED)
@pytest.mark.parametrize("dt", [BF, FP])
def test_grouped(moe, counts, K, N, first, behind, dt):
    check_grouped(moe, counts, K, N, dt, first, behind, seed=len(counts))


@pytest.mark.parametrize("mean,K", [(2, 640), (3, 1152), (9, 896), (30, 640), (36, 1408), (60, 640)])
def test_grouped_several_tiles_per_block(moe, mean, K):
    """More tiles than SMs, of every kind, with numbers of blocks of 128 k that no batch or ring divides."""
    check_grouped(moe, np.random.default_rng(K).integers(0, 2 * mean + 1, 60).tolist(), K, 700, BF, first=1, behind=2, seed=mean)


def test_grouped_many_experts(moe):
    counts = np.random.default_rng(0).integers(0, 5, 1024).tolist()
    check_grouped(moe, counts, 128, 128, HF)
    check_grouped(moe, (np.random.default_rng(1).integers(0, 3, 1024) * 40).tolist(), 128, 96, BF, behind=10)


def test_grouped_equals_linear_rows(moe):
    """A row's result does not depend on the rows beside it within one plan: an expert's rows alone, moved."""
    K, N = 1024, 300
    a = check_grouped(moe, [40, 50, 30], K, N, FP, seed=2)
    assert torch.equal(a, check_grouped(moe, [40, 50, 30], K, N, FP, seed=2))


def test_products_past_32_bits(moe):
    """Weights past 2^32 codes, and outputs past 2^31 elements: the last experts, rows and channels."""
    E, N, K = 270, 4096, 4096
    wq = torch.randint(0, 0x7f, (E, N, K), dtype=torch.uint8, device="cuda").view(E4)
    ws = torch.full((E, N // B, K // B), 2.0 ** -12, device="cuda")
    for counts in ([0] * (E - 3) + [2, 0, 3], [0] * (E - 2) + [60, 200]):   # weights for few rows; with a mean of few, too
        offsets = torch.tensor([0, *np.cumsum(counts)], dtype=I32, device="cuda")
        n = int(offsets[-1])
        xq, xs = rows_f8(n, K, 3)
        out = moe.grouped_linear_f8(xq, xs, wq, ws, offsets, dtype=FP)
        for e in (E - 3, E - 2, E - 1):
            a, b = int(offsets[e]), int(offsets[e + 1])
            if a < b:
                ref, S = product_ref(xq[a:b], xs[a:b], wq[e], ws[e])
                check(out[a:b], ref, U, f"expert {e}", extra=product_tol(K, S))
    T, N, K = 70000, 32768, 128
    xq, xs = rows_f8(T, K, 5)
    w, s = rows_f8(N, K, 6)[0], torch.rand(N // B, 1, device="cuda")
    out = moe.linear_f8(xq, xs, w, s)
    for a in (0, 65500, T - 100):
        ref, S = product_ref(xq[a:a + 100], xs[a:a + 100], w, s)
        check(out[a:a + 100], ref, half_step(BF) + U, "linear", extra=product_tol(K, S))


@pytest.mark.parametrize("n", [12, 900])
def test_grouped_bad_offsets(moe, n):
    """Offsets out of order or out of range are taken as the nearest that are not, and show in the status."""
    K, N, E = 256, 130, 4
    xq, xs = rows_f8(n, K, 1)
    wq, ws = rows_f8(E * N, K, 2)[0].view(E, N, K), torch.full((E, 2, K // B), 0.001, device="cuda")
    status = torch.zeros(4, dtype=torch.uint8, device="cuda")
    for bad, good in (([-5, n // 3, n // 2, n, n], [0, n // 3, n // 2, n, n]), ([0, n // 2, n // 3, n, n + 100], [0, n // 2, n // 2, n, n]),
                      ([2 ** 31 - 1, -2 ** 31, 3, 2, 1], [n] * 5), ([0, 2 ** 31 - 1, 5, 6, 7], [0, n, n, n, n])):
        outs = []
        for off in (bad, good):
            out = torch.full((n, N), 3.0, dtype=BF, device="cuda")
            moe.grouped_linear_f8(xq, xs, wq, ws, torch.tensor(off, dtype=I32, device="cuda"), out=out, workspace=status)
            assert moe.read_status(status) == (moe.ERR_BAD_ROUTING if off is bad else moe.OK)
            outs.append(out)
        assert torch.equal(*outs)


# ---------------------------------------------------------------- weights to blocks


def check_blocks(q, s, w):
    w = w.double()
    E, N, K = w.shape
    pad = torch.zeros(E, -(-N // B) * B, K, dtype=torch.float64, device="cuda")
    pad[:, :N] = w
    m = pad.view(E, -1, B, K // B, B).abs().amax(dim=(2, 4))
    ref = torch.where(m < 2.0 ** -100, 0.0, m / 448)
    check(s, ref, 2 * U, "scales")
    by = ref.repeat_interleave(B, dim=1)[:, :N].repeat_interleave(B, dim=2)
    got = q.double() * s.double().repeat_interleave(B, dim=1)[:, :N].repeat_interleave(B, dim=2)
    half = torch.maximum(w.abs() * 2.0 ** -4, by * 2.0 ** -10) + 8 * U * w.abs()
    assert bool(((got - w).abs() <= half + 2.0 ** -99).all())


@pytest.mark.parametrize("E,N,K", [(1, 1, 128), (1, 128, 128), (2, 130, 256), (3, 127, 384), (1, 1000, 2048), (5, 300, 128), (2, 1, 512)])
@pytest.mark.parametrize("dt", [BF, HF, FP])
def test_blocks(moe, E, N, K, dt):
    w = (randn(E, N, K, seed=N) * torch.exp(randn(E, N, 1, seed=K))).to(dt)
    q, s = moe.quantize_blocks_f8(w)
    check_blocks(q, s, w)
    q2, s2 = moe.quantize_blocks_f8(w[0])
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])
    wide = torch.zeros(E, N + 1, K + 11, dtype=dt, device="cuda")
    wide[:, :N, 3:3 + K] = w                                    # rows off 16-byte boundaries
    q2, s2 = moe.quantize_blocks_f8(wide[:, :N, 3:3 + K])
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    for t in (w.transpose(1, 2).contiguous(), torch.nn.functional.pad(w.transpose(1, 2), (1, 4))[:, :, 1:N + 1]):
        q2, s2 = moe.quantize_blocks_f8(t.transpose(1, 2))      # columns contiguous
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    buf = torch.zeros(E * N * K + 5, dtype=torch.uint8, device="cuda")
    q2, _ = moe.quantize_blocks_f8(w, q=buf[3:3 + E * N * K].view(E4).view(E, N, K))
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and bool((buf[:3] == 0).all()) and bool((buf[-2:] == 0).all())


def test_blocks_edges(moe):
    w = randn(256, 384, seed=1)
    w[:128, :128] = 0.0
    w[:128, 128:256] = 2.0 ** -101
    w[130, 5], w[140, 130] = float("inf"), float("nan")
    w[128:, 256:] *= 1e30
    q, s = moe.quantize_blocks_f8(w)
    assert s[0, 0] == 0 and s[0, 1] == 0 and bool((q[:128, :256].float() == 0).all())
    assert not bool(s[1, 0].isfinite()) and not bool(s[1, 1].isfinite()) and bool((q[128:, :256].float() == 0).all())
    check_blocks(q[:, 256:][None].contiguous(), s[:, 2:][None].contiguous(), w[None, :, 256:])


def test_transposed_weight_gives_the_gradient(moe):
    """The rows' gradient is the product of the output's gradient with the transposed blocks: the same codes, and the
    product in 64 bits of the values."""
    N, K = 384, 256
    w = randn(N, K, seed=3, scale=0.05)
    q, s = moe.quantize_blocks_f8(w)
    qt, st = moe.quantize_blocks_f8(w.t())
    assert torch.equal(qt.t().float(), q.float()) and torch.equal(st.t(), s)
    d, ds = moe.quantize_q8(randn(50, N, seed=4), q_dtype=E4, group_size=B)
    dx = moe.linear_f8(d, ds, qt, st, dtype=FP)
    ref, S = values(d, ds) @ block_values(q, s), values(d, ds).abs() @ block_values(q, s).abs()
    check(dx, ref, U, "dx", extra=product_tol(N, S))


# ---------------------------------------------------------------- together


def f8_inputs(T, E=16, K=512, N=256, topk=4, seed=0, total=None):
    xq, xs = rows_f8(T, K, seed)
    xs = xs * 0.1
    w = torch.rand(T, topk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    wq = lambda n, k, s: quantized(E, n, k, s)  # noqa: E731
    return xq, xs, make_ids(T, topk, total or E, seed=seed), w, *wq(2 * N, K, seed + 1), *wq(K, N, seed + 2)


def quantized(E, N, K, seed):
    import wna16_grouped_gemm_gb300 as m
    return m.quantize_blocks_f8(randn(E, N, K, seed=seed, scale=K ** -0.5))


@pytest.mark.parametrize("T,begin", [(1, 0), (7, 0), (60, 8), (500, 0)])
def test_forward(moe, T, begin):
    """Against 64-bit products of the values that codes stand for.  The gate and the up products are rounded to bf16
    (2^-8 of g moves silu by at most 1.1 * 2^-8 |g|), h to e4m3 (half a step: 2^-4, or 2^-10 of its scale), y to bf16, and
    the sums have their own errors; what h's errors do to y is at most |W2| times them."""
    xq, xs, ids, w, w13, s13, w2, s2 = f8_inputs(T, seed=T, total=32 if begin else None)
    out = moe.forward_f8(xq, xs, ids, w, w13, s13, w2, s2, expert_begin=begin)
    x = values(xq, xs)
    ref, tol = torch.zeros(T, x.shape[1], dtype=torch.float64, device="cuda"), 0.0
    for e in range(w13.shape[0]):
        t, j = (ids == e + begin).nonzero(as_tuple=True)
        if not t.numel():
            continue
        W13, W2 = block_values(w13[e], s13[e]), block_values(w2[e], s2[e])
        g, u = (x[t] @ W13.t()).chunk(2, dim=1)
        dg, du = (product_tol(x.shape[1], x[t].abs() @ W13.abs().t()) + 2.0 ** -8 * (x[t] @ W13.t()).abs()).chunk(2, dim=1)
        g, u = g.clamp(max=7.0), u.clamp(-7.0, 7.0)
        silu = g / (1 + torch.exp(-g))
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 16 * U * h.abs()
        scale = (h.abs() + dh).view(t.numel(), -1, B).amax(dim=2).repeat_interleave(B, dim=1) / 448
        dh = dh + torch.maximum((h.abs() + dh) * 2.0 ** -4, scale * 2.0 ** -10) * 1.01
        y, S = h @ W2.t(), (h.abs() + dh) @ W2.abs().t()
        dy = dh @ W2.abs().t() + product_tol(h.shape[1], S)
        dy = dy + 2.0 ** -8 * (y.abs() + dy)
        wt = w[t, j].double().unsqueeze(1)
        ref.index_add_(0, t, wt * y)
        tol = tol + torch.zeros_like(ref).index_add_(0, t, wt * dy)
    check(out, ref, half_step(BF) + 8 * U, "forward", extra=1.01 * tol)
    # the parts, one by one, give the same bits
    rows, rs, off, inv = moe.sort_tokens(xq, ids, 16, scales=xs, expert_begin=begin)
    hq, hs = moe.swiglu_q8(moe.grouped_linear_f8(rows, rs, w13, s13, off), q_dtype=E4, group_size=B)
    assert torch.equal(out, moe.unsort_tokens(moe.grouped_linear_f8(hq, hs, w2, s2, off), inv, w))
    add = randn(T, x.shape[1], seed=9, dtype=BF)
    with_add = moe.forward_f8(xq, xs, ids, w, w13, s13, w2, s2, expert_begin=begin, addend=add)
    check(with_add, ref + add.double(), half_step(BF) + 8 * U, "forward", extra=1.01 * tol + 4 * U * add.double().abs())


def test_forward_without_rows(moe):
    """No token, and tokens none of whose experts are here."""
    xq, xs, ids, w, w13, s13, w2, s2 = f8_inputs(5, seed=1)
    assert moe.forward_f8(xq[:0], xs[:0], ids[:0], w[:0], w13, s13, w2, s2).shape == (0, 512)
    assert bool((moe.forward_f8(xq, xs, ids, w, w13, s13, w2, s2, expert_begin=100) == 0).all())
    add = randn(5, 512, dtype=BF)
    assert torch.equal(moe.forward_f8(xq, xs, ids, w, w13, s13, w2, s2, expert_begin=100, addend=add), add)


def test_forward_expert_ranges_add_up(moe):
    """Two halves of the experts, the second with the first's output as its addend: one more rounding (2^-8 of what the first gives)."""
    xq, xs, ids, w, w13, s13, w2, s2 = f8_inputs(40, seed=3)
    whole = moe.forward_f8(xq, xs, ids, w, w13, s13, w2, s2, dtype=FP)
    half = moe.forward_f8(xq, xs, ids, w, w13[:8], s13[:8], w2[:8], s2[:8], dtype=FP)
    both = moe.forward_f8(xq, xs, ids, w, w13[8:], s13[8:], w2[8:], s2[8:], expert_begin=8, addend=half, dtype=FP)
    assert both.dtype == FP and float((both - whole).norm()) <= 8 * U * float(whole.norm() + half.norm()) * 4


def _block(moe, T, shared_f8, routed_f8, seed=0):
    from tests.test_gpu_block import _block_inputs
    x, r, w, kw = _block_inputs(T, seed=seed)
    if shared_f8:
        w.shared_w13, w.shared_w13_scales = moe.quantize_blocks_f8(randn(768, 512, seed=1, scale=512 ** -0.5))
        w.shared_w2, w.shared_w2_scales = moe.quantize_blocks_f8(randn(512, 384, seed=2, scale=384 ** -0.5))
    if routed_f8:
        w.w13_packed, w.w13_scales = quantized(8, 512, 512, 11)
        w.w2_packed, w.w2_scales = quantized(8, 512, 256, 12)
        kw = {k: v for k, v in kw.items() if k not in ("bits", "group_size")}
    return x, r, w, kw


@pytest.mark.parametrize("shared_f8,routed_f8", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("T", [1, 90, 600])
def test_moe_block(moe, T, shared_f8, routed_f8):
    """The block is its parts, bit for bit (each is tested by itself)."""
    x, r, w, kw = _block(moe, T, shared_f8, routed_f8)
    out, h = moe.moe_block(x, r, w, **kw)
    f8 = dict(q_dtype=E4, group_size=B)
    q, s, h2, n = moe.add_rmsnorm_q8(x, w.norm, r, want_norm=True)
    q8, s8 = moe.add_rmsnorm_q8(x, w.norm, r, **f8)[:2] if shared_f8 else moe.quantize_q8(n, **f8)
    ids, wt = moe.route_scored(n @ w.gate.t(), 2, bias=w.gate_bias, groups=4, topk_groups=2, scale=1.5)
    if routed_f8:
        ref = moe.forward_f8(q8, s8, ids, wt, w.w13_packed, w.w13_scales, w.w2_packed, w.w2_scales)
    else:
        ref = moe.forward(n, ids, wt, w.w13_packed, w.w13_scales, w.w2_packed, w.w2_scales, bits=4, group_size=128)
    if shared_f8:
        hq, hs = moe.swiglu_q8(moe.linear_f8(q8, s8, w.shared_w13, w.shared_w13_scales), **f8)
        ref = moe.linear_f8(hq, hs, w.shared_w2, w.shared_w2_scales, addend=ref)
    else:
        hq, hs = moe.swiglu_q8(moe.linear_q8(q, s, w.shared_w13, w.shared_w13_scales))
        ref = moe.linear_q8(hq, hs, w.shared_w2, w.shared_w2_scales, addend=ref)
    assert torch.equal(out, ref) and torch.equal(h, h2)


def test_moe_block_needs_the_sizes_of_wna16_experts(moe):
    x, r, w, kw = _block(moe, 2, True, False)
    with pytest.raises(TypeError, match="bits"):
        moe.moe_block(x, r, w, topk=2)


@pytest.mark.parametrize("T", [3, 60, 1200])
def test_other_stream_and_graph(moe, T):
    """On a side stream, and replayed from a graph with new inputs and other routing: the bits of the eager call."""
    x, r, w, kw = _block(moe, T, True, True)
    out, res = moe.moe_block(x, r, w, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, r2 = moe.moe_block(x, r, w, **kw)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(res, r2)
    sx, sr = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gr = moe.moe_block(sx, sr, w, **kw)
    for seed in (11, 12):
        sx.copy_(randn(*x.shape, seed=seed, dtype=BF))
        sr.copy_(randn(*x.shape, seed=seed + 5, dtype=BF))
        graph.replay()
        eo, er = moe.moe_block(sx, sr, w, **kw)
        torch.cuda.synchronize()
        assert torch.equal(go, eo) and torch.equal(gr, er)


@pytest.mark.parametrize("T", [300, 4000])
def test_backward_in_a_graph(moe, T):
    """The gradients, captured and replayed, while an eager result of the same tensors lives."""
    topk, E, K = 4, 16, 512
    ids, w = make_ids(T, topk, E), torch.rand(T, topk, device="cuda")
    x, d = randn(T, K, dtype=BF), randn(T, K, seed=1, dtype=BF)

    def back():
        rows, _, _, inv = moe.sort_tokens(x, ids, E)
        dy, dw = moe.unsort_tokens_grad(d, inv, rows, w)
        return moe.unsort_tokens(dy, inv), dw

    alive = back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = back()
    for seed in (3, 4):
        x.copy_(randn(T, K, seed=seed, dtype=BF))
        ids.copy_(make_ids(T, topk, E, seed=seed))
        graph.replay()
        ref = back()
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert torch.equal(alive[0], got[0]) and not torch.equal(alive[1], got[1])   # dx is dout times the sum of the weights


def test_two_streams_at_once(moe):
    """Calls that run at the same time share nothing (each has its own status word, or none)."""
    cases = [(4, 2048, 512), (150, 1024, 768), (900, 512, 1024)]
    want = [check_linear(moe, *c, FP, seed=c[0]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                T, K, N = c
                xq, xs = rows_f8(T, K, T)
                got.append(moe.linear_f8(xq, xs, rows_f8(N, K, T + 10)[0], torch.exp(randn(-(-N // B), K // B, seed=T + 12)) * 0.001, dtype=FP))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs_at_once(moe):
    """Two captured layers, replayed at the same time on two streams, share nothing."""
    graphs, got, want = [], [], []
    for T in (30, 2500):
        xq, xs, ids, w, w13, s13, w2, s2 = f8_inputs(T, seed=T)
        want.append(moe.forward_f8(xq, xs, ids, w, w13, s13, w2, s2))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = moe.forward_f8(xq, xs, ids, w, w13, s13, w2, s2)
        graphs.append((g, xq, xs, ids, w, w13, s13, w2, s2))
        got.append(out)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_debug_build_matches_release(moe):
    """The bounds-checked build gives the same bits."""
    from wna16_grouped_gemm_gb300 import binding, build, f8
    build.build(debug=True)
    saved = f8._load()
    outs = []
    try:
        for entries in (saved, f8.declare(binding.load_debug_library())):
            f8._entries = entries
            outs.append([check_linear(moe, 7, 512, 50, FP), check_linear(moe, 70, 1024, 130, FP), check_linear(moe, 600, 2048, 1024, FP),
                         check_grouped(moe, [3, 0, 40, 200], 512, 300, FP), check_sort(moe, randn(700, 128), make_ids(700, 8, 64), 64)[0]])
    finally:
        f8._entries = saved
    for a, b in zip(*outs):
        assert torch.equal(a, b)
