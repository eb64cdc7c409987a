"""The operators around the routed experts on the GPU at the edges of their
ranges, against plain 64-bit computations of their definitions (tolerances:
as derived in test_gpu_block, u = 2^-24)."""
from __future__ import annotations

import ctypes
import dataclasses
import itertools

import numpy as np
import pytest
import torch

from tests.test_gpu_block import (_block_inputs, BF, FP, HF, I8, U, check, check_q8, check_route, half_step, moe, norm_ref,  # noqa: F401
                                  randn, route_ref)

pytestmark = pytest.mark.gpu

INF = float("inf")


# ---------------------------------------------------------------- norm


def _norm_c(x, r, w, q, s, ro, no, group=0, eps=1e-6):
    """The C entry point itself; None: NULL."""
    from wna16_grouped_gemm_gb300 import block
    lib = block._load()
    types = {BF: 0, HF: 1, FP: 2}
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    T, K = x.shape
    return lib.wna16_moe_add_rmsnorm_q8(p(x), K, p(r), K, p(w), types[w.dtype], T, K, types[x.dtype], eps, 0, group, p(q), p(s),
                                        p(ro), p(no), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


@pytest.mark.parametrize("T,K,dt,group", [(5, 264, BF, 0), (3, 1003, BF, 0), (700, 512, HF, 64), (4, 640, FP, 128), (2, 9000, FP, 0)])
def test_norm_with_every_choice_of_outputs(moe, T, K, dt, group):
    """Each of residual, residual_out, norm_out and (q, scales) may be NULL by itself;
    what is written has the bits that it has with all of them."""
    x, w = randn(T, K, seed=1, dtype=dt), (1 + 0.2 * randn(K, seed=2)).to(dt)
    for r in (None, randn(T, K, seed=3, dtype=dt)):
        h, y = norm_ref(x, w, r, 1e-6)
        full = None
        for has_ro, has_no, has_q in itertools.product((True, False), repeat=3):
            ro = torch.full_like(x, 77.0) if has_ro else None
            no = torch.full_like(x, 77.0) if has_no else None
            q = torch.full((T, K), 77, dtype=I8, device="cuda") if has_q else None
            s = torch.full((T, K // group if group else 1), 77.0, device="cuda") if has_q else None
            rc = _norm_c(x, r, w, q, s, ro, no, group)
            if not has_no and not has_q:
                assert rc == moe.ERR_INVALID_ARG
                continue
            assert rc == moe.OK
            torch.cuda.synchronize()
            if full is None:
                full = ro, no, q, s
                if r is None:
                    assert torch.equal(ro, x)
                else:
                    check(ro, h, half_step(dt) + 2 * U, "residual_out")
                check(no, y, half_step(dt) + 33 * U, "norm_out", floor=2.0 ** -25 if dt == HF else 0.0)
                check_q8(moe, q, s, y, group, 32 * U, "norm")
            for got, want in zip((ro, no, q, s), full):
                assert got is None or torch.equal(got, want), (has_ro, has_no, has_q)


def test_norm_residual_out_without_a_residual(moe):
    x, w = randn(6, 512, seed=4, dtype=BF), torch.ones(512, dtype=BF, device="cuda")
    ro = torch.zeros_like(x)
    q, s, got, _ = moe.add_rmsnorm_q8(x, w, residual_out=ro)
    assert got is ro and torch.equal(ro, x)
    q2, s2, none, _ = moe.add_rmsnorm_q8(x, w)
    assert none is None and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("qt", [I8, torch.float8_e4m3fn])
def test_norm_of_tiny_rows(moe, qt, group):
    """Rows that the norm makes large again (a small eps): right as far as their codes can be made in
    fp32, zeros below that, and never the codes of an infinite factor."""
    x = randn(6, 256, seed=5)
    for t, size in enumerate((1e-20, 1e-30, 1e-33, 5e-36, 1e-38, 1e-44)):
        x[t] *= size
    w = torch.ones(256, device="cuda")
    q, s, _, no = moe.add_rmsnorm_q8(x, w, eps=1e-30, q_dtype=qt, group_size=group, want_norm=True)
    _, y = norm_ref(x, w, None, float(torch.tensor(1e-30)))
    check(no[:4], y[:4], 33 * U, "norm_out")
    check_q8(moe, q[:4], s[:4], y[:4], group, 32 * U, "tiny")
    assert not bool(s[4:].any()) and not bool(moe.dequantize_q8(q[4:], s[4:], dtype=FP).any())


# ---------------------------------------------------------------- routing


def _group_bias(E, G, groups, value, seed=0):
    """A small bias, and `value` for the experts of the given groups."""
    b = randn(E, seed=seed, scale=0.02)
    b.view(G, E // G)[groups] = value
    return b


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("gscore", ["max", "top2"])
@pytest.mark.parametrize("E,G,Gk", [(256, 8, 4), (36, 12, 5), (1020, 17, 6), (160, 8, 3)])
def test_route_groups_masked_by_the_lowest_bias(moe, score, gscore, E, G, Gk):
    """Groups with a bias of fp32's lowest value: fewer groups than are kept stay
    unmasked, as many, one, none.  (Group sizes that leave lanes with empty slots.)"""
    logits = randn(50, E, seed=E, scale=1.5)
    for left in (Gk + 1, Gk, Gk - 1, 1, 0):
        b = _group_bias(E, G, list(range(left, G)), torch.finfo(FP).min)
        for k in (1, 6, min(32, Gk * (E // G))):
            check_route(moe, logits, k, score=score, bias=b, G=G, Gk=Gk, group_score=gscore)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("gscore", ["max", "top2"])
@pytest.mark.parametrize("E,G,Gk", [(256, 8, 4), (36, 12, 5), (160, 8, 3)])
@pytest.mark.parametrize("value", [-1e9, -100.0, 1e9])
def test_route_groups_far_from_the_others(moe, score, gscore, E, G, Gk, value):
    """Groups masked or forced by a large bias: each group's score has an error of its own size."""
    logits = randn(60, E, seed=E + 1, scale=1.5)
    for left in (G - 1, Gk + 1, Gk, Gk - 1, 1):
        b = _group_bias(E, G, list(range(left, G)), value)
        for k in (1, 6, min(32, Gk * (E // G))):
            check_route(moe, logits, k, score=score, bias=b, G=G, Gk=Gk, group_score=gscore)
        b.view(G, E // G)[left:, 1:] = -value                       # one expert far up, the others far down, and the reverse
        check_route(moe, logits, 6, score=score, bias=b, G=G, Gk=Gk, group_score=gscore)


def _us(f, n=20):
    """Time of one call among others (median of five runs of a graph of n)."""
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            f()
    graph.replay()
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / n)
    return sorted(times)[2]


def test_route_groups_far_from_the_others_cost_no_64_bits(moe):
    """Masked groups leave the others' order as clear as it was: no token is chosen in 64 bits for
    them, which would take a hundred times as long."""
    logits, b = randn(8192, 256, seed=1), randn(256, seed=2, scale=0.05)
    ids, w = moe.route_scored(logits, 8, bias=b, groups=8, topk_groups=4)
    time = lambda bias: _us(lambda: moe.route_scored(logits, 8, bias=bias, groups=8, topk_groups=4, ids=ids, weights=w))  # noqa: E731
    plain = time(b)
    for value in (-1e9, torch.finfo(FP).min):
        for left in (7, 5, 4):
            masked = b.clone()
            masked.view(8, 32)[left:] = value
            assert time(masked) < 3 * plain, (value, left)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,Gk,k", [(256, 1, 1, 8), (256, 8, 4, 8), (1024, 1, 1, 32), (64, 1, 1, 31), (37, 1, 1, 5)])
def test_route_forced_and_masked_experts(moe, score, E, G, Gk, k):
    """Experts with large biases: neighbours are compared by their own size."""
    logits = randn(60, E, seed=E + k, scale=1.5)
    for value in (1e9, -1e9, 1e4, torch.finfo(FP).max, torch.finfo(FP).min):
        for n in (1, 2, k - 1, E // 2):
            b = randn(E, seed=n, scale=0.05)
            b[torch.randperm(E, generator=torch.Generator().manual_seed(n))[:n].cuda()] = value
            check_route(moe, logits, k, score=score, bias=b, G=G, Gk=Gk)
    b = randn(E, seed=3, scale=0.05)
    b[:6] = torch.tensor([1e9, 1e9, 1e5, 1e5 + 0.0078125, -1e9, -1e30], device="cuda")   # pairs that 32 bits cannot order
    check_route(moe, logits, k, score=score, bias=b, G=G, Gk=Gk)


def test_route_forced_experts_cost_no_64_bits(moe):
    logits = randn(8192, 256, seed=1)
    ids, w = moe.route_scored(logits, 8)
    time = lambda bias: _us(lambda: moe.route_scored(logits, 8, bias=bias, ids=ids, weights=w))  # noqa: E731
    b = randn(256, seed=2, scale=0.05)
    plain = time(b)
    for value in (1e9, torch.finfo(FP).max):
        forced = b.clone()
        forced[5] = value
        assert time(forced) < 3 * plain, value


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,Gk", [(64, 1, 1), (256, 8, 4), (36, 12, 5), (1020, 17, 6), (1024, 1, 1)])
def test_route_bias_that_is_not_finite(moe, score, E, G, Gk):
    """NaN and infinities count as the nearest finite numbers, NaN as the lowest: the choice is
    always of topk experts there are."""
    inf, nan = float("inf"), float("nan")
    top = torch.finfo(FP).max
    logits = randn(40, E, seed=E + G, scale=1.5)
    base = randn(E, seed=E, scale=0.02)
    biases = [torch.full_like(base, v) for v in (nan, -inf, inf)]
    for n in (1, 3, E // 2, E - 2):
        at = torch.randperm(E, generator=torch.Generator().manual_seed(n))[:n].cuda()
        for v in (nan, -inf, inf):
            b = base.clone()
            b[at] = v
            biases.append(b)
    b = base.clone()
    b.view(G, E // G)[: (G + 1) // 2, 1:] = -inf                     # groups with one expert left
    biases.append(b)
    mixed = base.clone()
    mixed[0::4], mixed[1::4], mixed[2::4] = nan, -inf, inf
    biases.append(mixed)
    for b in biases:
        clean = torch.where(torch.isnan(b), -top, b).clamp(-top, top)
        for k, group_score in itertools.product((1, 5, min(32, Gk * (E // G))), ("max", "top2")):
            ids, w = check_route(moe, logits, k, score=score, bias=clean, G=G, Gk=Gk, group_score=group_score)
            got = moe.route_scored(logits, k, score=score, bias=b, groups=G, topk_groups=Gk, group_score=group_score)
            assert torch.equal(got[0].cpu(), torch.from_numpy(ids)) and torch.equal(got[1].double().cpu(), torch.from_numpy(w))


@pytest.mark.parametrize("dt", [FP, BF, HF])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("gscore", ["top2", "max"])
def test_route_infinite_logits_in_groups_that_lose(moe, dt, score, gscore):
    """A logit of +inf does not bring its expert back from a group that was not kept."""
    T, E, G = 24, 64, 8
    logits = randn(T, E, seed=12, dtype=dt)
    logits.view(T, G, -1)[:, 2:5] += 4.0                            # three good groups
    logits[:, 0:8] = -9.0
    logits[0::3, 3] = INF                                           # top2: 1 + 1e-4 against 1.9
    logits[1::3, 48:50] = INF
    logits[2::3, [1, 9, 17, 33, 41, 57]] = INF                      # in more groups than are kept
    logits[5::6, 20] = -INF
    for Gk in (1, 2, 3, 5):
        for k in (1, 4, 8):
            for renorm in (False, True):
                check_route(moe, logits, k, score=score, G=G, Gk=Gk, group_score=gscore, renorm=renorm)
    wide = randn(T, 1024, seed=13, dtype=dt)
    wide[:, 5] = INF
    wide[:, 0:5], wide[:, 6:64] = -9.0, -9.0
    wide[:, 64:200] = 2.0                                           # many equal values: one maximum per choice
    check_route(moe, wide, 32, score=score, G=16, Gk=2, group_score=gscore)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("centre", [-86.0, -88.5, -95.0, -104.0, -200.0, -690.0])
def test_route_weights_of_sigmoids_below_the_smallest(moe, bias, centre):
    """Weights divided by their sum keep the scores' ratios where the scores have left fp32."""
    T, E, k = 40, 64, 6
    logits = centre + randn(T, E, seed=7)
    logits[0:5, 3] = -5.0                                           # one well above the others
    logits[5:10, 3] = 2.0
    logits[10:15, 1::2] = -INF
    logits[15:18] = torch.finfo(FP).min                             # masked: weights 0
    b = randn(E, seed=8, scale=0.05) if bias else None
    ids, w = check_route(moe, logits, k, bias=b, scale=2.5)
    live = (ids >= 0) & (logits.cpu().gather(1, torch.from_numpy(ids)) > -1000).numpy()
    for t in range(T):
        if live[t].any():
            assert abs(w[t].sum() / 2.5 - 1) < 1e-5
        assert not w[t][~live[t]].any()
    # without the division: below 2^-126 in steps of 2^-149 (times the scale, which is below 3)
    _, rw = route_ref(logits, k, "sigmoid", b, 1, 1, "top2", False, 2.5)
    _, got = moe.route_scored(logits, k, bias=b, renormalize=False, scale=2.5)
    assert bool((torch.from_numpy(rw) - got.double().cpu()).abs().le(256 * U * torch.from_numpy(rw) + 4 * 2.0 ** -149).all())


@pytest.mark.parametrize("dt", [FP, BF, HF])
def test_route_masked_experts_that_a_bias_chooses(moe, dt):
    """Experts masked by their type's lowest value, or by -30000, and chosen all the same score 0: they
    share no weight, alone or beside one that is not masked."""
    logits = randn(30, 32, seed=5, dtype=dt)
    bias = torch.zeros(32, device="cuda")
    bias[8:16] = 4.0
    for score in ("softmax", "sigmoid"):
        for mask in (-30000.0, torch.finfo(dt).min, -INF):
            z = logits.clone()
            z[:, 8:16] = mask
            z[::3, 11] = 0.5
            for k in (1, 4, 8):
                for G, Gk in ((1, 1), (4, 1)):
                    ids, w = check_route(moe, z, k, score=score, bias=bias, G=G, Gk=Gk)
                    live = (ids == 11) & (np.arange(30) % 3 == 0)[:, None]
                    assert not w[~live].any() and np.abs(w[live] - 1).max() < 1e-6


# ---------------------------------------------------------------- the block


def test_moe_block_without_a_residual(moe):
    """h = x: the output of a residual of zeros, and x as the next block's residual."""
    x, r, w, kw = _block_inputs(37)
    out, h = moe.moe_block(x, None, w, **kw)
    same, h0 = moe.moe_block(x, torch.zeros_like(r), w, **kw)
    assert torch.equal(out, same) and torch.equal(h, x) and torch.equal(h0, x)
    moe.moe_block(out, h, w, **kw)                                  # the next one takes it


def test_moe_block_with_an_fp32_gate(moe):
    """The choice is that of fp32 logits: the block has the bits of its parts with them, and experts
    that differ by less than bf16 can tell are told apart."""
    x, r, w, kw = _block_inputs(300)
    gate = w.gate.float()
    gate[1::2] = gate[0::2] * (1 + 2.0 ** -12)                      # pairs whose logits agree to 12 bits
    w = dataclasses.replace(w, gate=gate, gate_bias=None)
    kw = dict(kw, groups=1, topk_groups=1)
    out, h = moe.moe_block(x, r, w, **kw)
    q, s, res, normed = moe.add_rmsnorm_q8(x, w.norm, r, want_norm=True)
    ids, wts = moe.route_scored(normed.float() @ gate.t(), kw["topk"], scale=kw["scale"])
    routed = moe.forward(normed, ids, wts, w.w13_packed, w.w13_scales, w.w2_packed, w.w2_scales, bits=4, group_size=128)
    hq, hs = moe.swiglu_q8(moe.linear_q8(q, s, w.shared_w13, w.shared_w13_scales, dtype=x.dtype))
    assert torch.equal(out, moe.linear_q8(hq, hs, w.shared_w2, w.shared_w2_scales, addend=routed)) and torch.equal(h, res)
    exact = normed.double() @ gate.double().t()
    best = exact.max(dim=1, keepdim=True).values                    # (fp32 sums of 512 terms: 1e-5 of them)
    assert bool(((best - exact.gather(1, ids[:, :1].long())).abs() <= 1e-4 * best.abs()).all())
    far = (best[:, 0].abs() > 0.5) & (exact.gather(1, ids[:, :1].long() ^ 1) < best)[:, 0]
    assert int(far.sum()) > 100 and bool((exact.argmax(dim=1) == ids[:, 0].long())[far].all())


# ---------------------------------------------------------------- linear


@pytest.mark.parametrize("T", [4, 64, 600, 2048])
@pytest.mark.parametrize("K", [1024, 4096, 65536])
def test_linear_large_sums_that_cancel(moe, T, K):
    """Partial sums far above 2^24 that cancel to small ones, and long tails of small products behind
    them.  Up to 32 tokens and up to 1024 k the sums are exact; else they are off by at most 2^-20 of
    the sum of the products' magnitudes per 16 k, whatever is left of it."""
    N, h = 512, K // 2
    g = torch.Generator(device="cuda")
    g.manual_seed(K + T)
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int16).to(I8)  # noqa: E731
    big = torch.full((T, K), 127, dtype=I8, device="cuda"), torch.full((N, K), 127, dtype=I8, device="cuda")
    x, w = r(100, 128, T, K), r(100, 128, N, K)
    x[:, h:], w[:, h:] = -x[:, :h], w[:, :h]
    x[:, -16:] = r(-128, 128, T, 16)                                # all that is left
    tail = big[0].clone(), big[1].clone()
    tail[0][:, h:], tail[1][:, h:] = 31, 33
    down = big[0].clone(), big[1]
    down[0][:, h:] = -3
    for xq, wq in ((x, w), tail, down):
        S = xq.double().abs() @ wq.double().abs().t()
        ref = xq.double() @ wq.double().t()
        out = moe.linear_q8(xq, torch.ones(T, device="cuda"), wq, torch.ones(N, device="cuda"), dtype=FP).double()
        tol = 0.0 if T <= 32 or K <= 1024 else K / 16 * 2.0 ** -20 * S
        assert bool(((out - ref).abs() <= U * ref.abs() + tol).all()), float(((out - ref).abs() / S).max())


@pytest.mark.parametrize("T", [1, 32, 33, 600])
def test_linear_status_for_any_number_of_tokens(moe, T):
    """A workspace that is kept for larger batches holds this call's status, not what was there."""
    K, N = 512, 384
    ws = torch.full((256,), 0x5a, dtype=torch.uint8, device="cuda")
    xq, wq = torch.ones(T, K, dtype=I8, device="cuda"), torch.ones(N, K, dtype=I8, device="cuda")
    out = moe.linear_q8(xq, torch.ones(T, device="cuda"), wq, torch.ones(N, device="cuda"), workspace=ws, dtype=FP)
    assert bool((out == K).all())
    assert moe.read_status(ws) == moe.OK
    assert bool((ws[4:] == 0x5a).all())
    if T <= 32:                                                     # none is needed
        for small in (ws[:0], ws[:3], ws[1:9], ws[8:16]):
            again = moe.linear_q8(xq, torch.ones(T, device="cuda"), wq, torch.ones(N, device="cuda"), workspace=small, dtype=FP)
            assert torch.equal(out, again)
        assert bool((ws[16:] == 0x5a).all())
