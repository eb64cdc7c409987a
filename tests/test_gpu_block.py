"""The operators around the routed experts on the GPU, against plain 64-bit
computations of their definitions.

Tolerances, with u = 2^-24 (fp32 half step) and e = eps(type) / 2 (the output's
half step):
  norm    h is one fp32 addition (u); the sum of squares is at most 32 serial and
          10 tree additions of positive terms, halved by the root (21 u), the mean,
          eps, rsqrtf (2 ulp) and two products add 8 u: y within 32 u of itself.
  scales  y's maximum, one division: 34 u.
  values  code * scale in fp32: the rounding to a code is off by half a step, the
          quotient before it by 36 u of at most 127 steps, the scale by 34 u:
          scale * (0.5 + 127 * 72 u) for int8; e4m3: half a step is 2^-4 of the
          value or 2^-10 scale, and 72 u of it.
  swiglu  expf (2 ulp), the sum, the division and the product: 12 u in y's place.
  linear  exact integer sum; the conversion, two products, bias and addend: 5 u of
          the magnitudes added; then the output's rounding.
  route   experts exact; weights: a sigmoid's 5 u or a softmax's 60 u + its sum's
          2 * 64 u, the sum of the chosen, a division and a product: 256 u.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
I8, E4 = torch.int8, torch.float8_e4m3fn
Q = {I8: 127.0, E4: 448.0}


@pytest.fixture(scope="module")
def moe():
    import wna16_grouped_gemm_gb300 as m
    from wna16_grouped_gemm_gb300 import build
    build.build()
    m.load_library()
    return m


def half_step(dt):
    return torch.finfo(dt).eps / 2


def randn(*shape, seed=0, dtype=FP, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def check(got, ref, rel, what, floor=0.0, extra=0.0):
    """|got - ref| <= rel |ref| + extra + floor, elementwise, NaN where ref is."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    d = (got - ref).abs()
    bad = d > rel * ref.abs() + extra + floor
    worst = float((d / (ref.abs() + 1e-300)).nan_to_num(0, 0, 0).max()) if d.numel() else 0.0
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst relative {worst:.3g}"


def check_q8(moe, q, scales, y, group, dy, what):
    """q, scales against the 64-bit rows y; dy: y's own relative error in the kernel."""
    T, K = y.shape
    g = group or K
    m = y.view(T, K // g, g).abs().amax(dim=2)
    ref = torch.where(m < 2.0 ** -100, torch.zeros_like(m), m / Q[q.dtype])
    check(scales, ref, dy + 2 * U, what + " scales")
    if q.dtype == I8:
        assert int(q.min()) >= -127, what
    values = moe.dequantize_q8(q, scales, dtype=FP).double()
    s = ref.repeat_interleave(g, dim=1)
    slack = 2 * (dy + 4 * U)
    half = s * (0.5 + 127 * slack) if q.dtype == I8 else torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10) + 2 * slack * y.abs()
    d = (values - y).abs()
    assert not bool((d > half + 2.0 ** -99).any()), f"{what} values: worst {float((d / (s + 1e-300)).max()):.4f} steps"


def norm_ref(x, w, r, eps):
    h = x.double() if r is None else x.double() + r.double()
    return h, h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps) * w.double()


NORM_CASES = [
    # T, K, type, weight type, residual, q type, group
    (1, 4096, BF, BF, True, I8, 0), (4, 4096, BF, FP, True, I8, 0), (33, 4096, BF, BF, True, E4, 128),
    (7, 2048, HF, HF, True, I8, 64), (5, 2056, BF, BF, True, I8, 0), (300, 5120, BF, BF, False, E4, 32),
    (3, 8192, FP, FP, True, I8, 256), (2, 16384, HF, FP, True, I8, 128), (2, 32768, BF, BF, True, I8, 0),
    (9, 1, BF, BF, True, I8, 0), (9, 3, HF, HF, False, E4, 0), (11, 1021, BF, BF, True, I8, 0),
    (6, 4097, FP, FP, True, E4, 0), (3, 24577, BF, FP, True, I8, 0), (17, 32, BF, BF, True, E4, 32),
    (2500, 96, BF, BF, True, I8, 32),
    # more rows than are worked on at the same time, and the sizes with two and four chunks per thread
    (3000, 4096, BF, BF, True, I8, 0), (512, 4096, BF, BF, True, I8, 0), (1500, 8192, HF, HF, False, E4, 64),
    (700, 12288, BF, BF, True, I8, 256),
]


@pytest.mark.parametrize("T,K,dt,wdt,res,qt,group", NORM_CASES)
def test_norm(moe, T, K, dt, wdt, res, qt, group):
    x, r = randn(T, K, seed=K, dtype=dt), randn(T, K, seed=K + 1, dtype=dt, scale=3.0) if res else None
    w = (1 + 0.2 * randn(K, seed=K + 2)).to(wdt)
    q, s, ro, no = moe.add_rmsnorm_q8(x, w, r, q_dtype=qt, group_size=group, want_norm=True)
    h, y = norm_ref(x, w, r, 1e-6)
    if res:
        check(ro, h, half_step(dt) + 2 * U, "residual")
    else:
        assert ro is None
    check(no, y, half_step(dt) + 33 * U, "norm", floor=2.0 ** -25 if dt == HF else 0.0)
    check_q8(moe, q, s, y, group, 32 * U, "norm")


def test_norm_strided_unaligned_and_in_place(moe):
    """Rows of a wider tensor, rows that start off 16-byte boundaries, and the
    residual updated in place."""
    T, K = 37, 1000
    w = (1 + 0.2 * randn(K, seed=1)).to(BF)
    for off, width in ((0, 1024), (8, 1016), (1, 1003), (3, 1008)):
        x = randn(T, width, seed=off, dtype=BF)[:, off:off + K]
        r = randn(T, width, seed=off + 9, dtype=BF)[:, off:off + K]
        q, s, ro, no = moe.add_rmsnorm_q8(x, w, r, want_norm=True)
        h, y = norm_ref(x, w, r, 1e-6)
        check(ro, h, half_step(BF) + 2 * U, f"residual {off}")
        check(no, y, half_step(BF) + 33 * U, f"norm {off}")
        check_q8(moe, q, s, y, 0, 32 * U, f"norm {off}")
    for K in (1000, 1003):
        w = (1 + 0.2 * randn(K, seed=1)).to(BF)
        x, r = randn(T, K, seed=5, dtype=BF), randn(T, K, seed=6, dtype=BF)
        q0, s0, ro0, no0 = moe.add_rmsnorm_q8(x, w, r, want_norm=True)
        r2 = r.clone()
        q1, s1, ro1, no1 = moe.add_rmsnorm_q8(x, w, r2, want_norm=True, residual_out=r2)
        assert ro1 is r2
        x2 = x.clone()
        q2, s2, ro2, _ = moe.add_rmsnorm_q8(x2, w, r, residual_out=x2)
        for a, b in ((q0, q1), (s0, s1), (ro0, ro1), (no0, no1), (q0, q2), (s0, s2), (ro0, ro2)):
            assert torch.equal(a, b)


def test_norm_parts(moe):
    """16-bit output alone, 8-bit output alone, no residual: the same bits as all together."""
    x, r, w = randn(20, 4096, dtype=BF), randn(20, 4096, seed=1, dtype=BF), randn(4096, seed=2, dtype=BF)
    q, s, ro, no = moe.add_rmsnorm_q8(x, w, r, want_norm=True)
    a = moe.add_rmsnorm_q8(x, w, r, want_q=False, want_norm=True)
    assert a[0] is None and a[1] is None and torch.equal(a[3], no) and torch.equal(a[2], ro)
    b = moe.add_rmsnorm_q8(x, w, r)
    assert b[3] is None and torch.equal(b[0], q) and torch.equal(b[1], s)
    with pytest.raises(moe.Wna16Error):
        moe.add_rmsnorm_q8(x, w, r, want_q=False)


def test_rows_without_a_scale(moe):
    """Zero rows, rows of tiny values, rows with NaN and infinities."""
    x = randn(6, 256, dtype=FP)
    x[0] = 0.0
    x[1] = 2.0 ** -110
    x[2, 17] = float("nan")
    x[3, 200] = float("inf")
    x[4] *= 2.0 ** -90
    for qt in (I8, E4):
        q, s = moe.quantize_q8(x, q_dtype=qt)
        v = moe.dequantize_q8(q, s, dtype=FP)
        assert not bool(s[:2].any()) and not bool(v[:2].any())
        assert not bool(torch.isfinite(s[2:4]).any()) and bool(torch.isnan(v[2:4]).all())
        check_q8(moe, q[4:], s[4:], x[4:].double(), 0, 0.0, str(qt))
        q, s = moe.quantize_q8(x, q_dtype=qt, group_size=64)      # only the run that holds it
        v = moe.dequantize_q8(q, s, dtype=FP)
        assert bool(torch.isnan(v[2, :64]).all()) and bool(torch.isfinite(v[2, 64:]).all())
        assert bool(torch.isnan(v[3, 192:]).all()) and bool(torch.isfinite(v[3, :192]).all())
    w = torch.ones(256, device="cuda")
    _, s, _, no = moe.add_rmsnorm_q8(x, w, want_norm=True)
    assert bool(torch.isnan(no[2]).all()) and not bool(torch.isfinite(s[2:4]).any())
    assert not bool(no[0].any()) and not bool(s[0].any())          # 0 / sqrt(eps)


@pytest.mark.parametrize("T,N,dt,L,qt,group", [
    (1, 2048, BF, 7.0, I8, 0), (4, 2048, BF, 7.0, E4, 128), (33, 512, HF, 7.0, I8, 64), (5, 1001, BF, 7.0, I8, 0),
    (3, 9000, FP, float("inf"), I8, 0), (700, 128, BF, 1.5, E4, 32), (2, 1, BF, 7.0, I8, 0), (2, 32768, BF, 7.0, I8, 0),
    (3000, 2048, BF, 7.0, I8, 0), (900, 12288, HF, 7.0, E4, 0), (40, 64, BF, float("inf"), E4, 64)])
def test_swiglu(moe, T, N, dt, L, qt, group):
    gu = randn(T, 2 * N, seed=N, dtype=dt, scale=4.0)
    gu[0, 0] = -200.0
    q, s = moe.swiglu_q8(gu, swiglu_limit=L, q_dtype=qt, group_size=group)
    g, up = gu.double().split(N, dim=1)
    g, up = g.clamp(max=L), up.clamp(-L, L)
    check_q8(moe, q, s, g / (1 + torch.exp(-g)) * up, group, 12 * U, "swiglu")
    wide = torch.zeros(T, 2 * N + 5, dtype=dt, device="cuda")
    wide[:, :2 * N] = gu
    q2, s2 = moe.swiglu_q8(wide[:, :2 * N], swiglu_limit=L, q_dtype=qt, group_size=group)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("L", [7.0, float("inf")])
def test_swiglu_over_the_range_of_gates(moe, dt, L):
    """One gate per row, from where the exponential overflows to where it vanishes."""
    g = torch.cat([torch.linspace(-130, 130, 1041), torch.tensor([-1e4, -1e30, -3e38, 1e4])]).to(dt).cuda()
    gu = torch.stack([g] * 8 + [torch.full_like(g, 3.0)] * 8, dim=1).contiguous()
    q, s = moe.swiglu_q8(gu, swiglu_limit=L)
    v = moe.dequantize_q8(q, s, dtype=FP).double()
    gd = g.double().clamp(max=L)
    ref = (gd * torch.sigmoid(gd) * 3.0)[:, None].expand(-1, 8)
    # the value's 12 roundings, of the scale 3, of the product 1; rows below 2^-100 are zeros
    assert bool(((v - ref).abs() <= 16 * U * ref.abs() + 2.0 ** -99).all())


def test_swiglu_nan_passes(moe):
    gu = randn(3, 64, dtype=BF)
    gu[0, 3] = float("nan")
    gu[1, 40] = float("nan")
    q, s = moe.swiglu_q8(gu)
    v = moe.dequantize_q8(q, s)
    assert bool(torch.isnan(v[:2]).all()) and bool(torch.isfinite(v[2]).all())


@pytest.mark.parametrize("K,group", [(4096, 0), (4096, 128), (37, 0), (5000, 0), (8192, 32)])
@pytest.mark.parametrize("dt", [BF, HF, FP])
@pytest.mark.parametrize("qt", [I8, E4])
def test_quantize_and_back(moe, K, group, dt, qt):
    x = randn(19, K, seed=K, dtype=dt)
    q, s = moe.quantize_q8(x, q_dtype=qt, group_size=group)
    check_q8(moe, q, s, x.double(), group, 0.0, "quantize")
    v = moe.dequantize_q8(q, s, dtype=dt)
    exact = q.double() * s.double().repeat_interleave(group or K, dim=1)
    check(v, exact, half_step(dt) + U, "dequantize", floor=2.0 ** -25 if dt == HF else 0.0)


def test_offsets_past_32_bits(moe):
    """2.2e9 codes: the last rows are as right as the first."""
    T, K = 540_000, 4096
    x = torch.zeros(T, K, dtype=BF, device="cuda")
    rows = [0, 1, T - 2, T - 1]
    x[rows] = randn(4, K, dtype=BF)
    q, s = moe.quantize_q8(x)
    v = moe.dequantize_q8(q, s)
    check_q8(moe, q[rows], s[rows], x[rows].double(), 0, 0.0, "long")
    check(v[rows], q[rows].double() * s[rows].double(), half_step(BF) + U, "long values")
    del x, q, s, v
    T, N, K = 70_000, 32_768, 64
    xq = torch.randint(-127, 128, (T, K), dtype=I8, device="cuda")
    wq = torch.randint(-127, 128, (N, K), dtype=I8, device="cuda")
    xs, ws = torch.rand(T, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    out = moe.linear_q8(xq, xs, wq, ws)
    ref = (xq[-40:].double() @ wq.double().t()) * xs[-40:, None].double() * ws.double()
    check(out[-40:], ref, half_step(BF) + 5 * U, "long linear")


# ---------------------------------------------------------------- routing


def route_ref(logits, k, score, bias, G, Gk, group_score, renorm, scale):
    z = logits.double().cpu().numpy()
    z = np.where(np.isnan(z), -np.inf, z)
    T, E = z.shape
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-z))
        else:
            m = z.max(axis=1, keepdims=True)
            e = np.where(z == m, 1.0, np.exp(z - m))
            s = np.where(np.isneginf(m), 0.0, e / e.sum(axis=1, keepdims=True))
    c = s if bias is None else s + bias.double().cpu().numpy()
    if Gk < G:
        g = np.sort(c.reshape(T, G, E // G), axis=2)
        gs = g[:, :, -1] if group_score == "max" or E // G < 2 else g[:, :, -1] + g[:, :, -2]
        keep = np.argsort(-gs, axis=1, kind="stable")[:, :Gk]
        mask = np.zeros((T, G), bool)
        np.put_along_axis(mask, keep, True, axis=1)
        c = np.where(np.repeat(mask, E // G, axis=1), c, -np.inf)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, axis=1)
    if renorm:
        t = w.sum(axis=1, keepdims=True)
        w = np.where(t > 0, w / np.where(t > 0, t, 1), 0)
    return ids, w * scale


def check_route(moe, logits, k, *, score="sigmoid", bias=None, G=1, Gk=1, group_score="top2", renorm=True, scale=1.0):
    ids, w = moe.route_scored(logits, k, score=score, bias=bias, groups=G, topk_groups=Gk, group_score=group_score,
                              renormalize=renorm, scale=scale)
    rid, rw = route_ref(logits, k, score, bias, G, Gk, group_score, renorm, scale)
    gid, gw = ids.cpu().numpy(), w.double().cpu().numpy()
    bad = np.flatnonzero((gid != rid).any(axis=1))
    assert bad.size == 0, f"{bad.size} tokens differ, first {bad[0]}: {gid[bad[0]]} for {rid[bad[0]]}"
    assert np.all(np.abs(gw - rw) <= 256 * U * np.abs(rw) + 1e-37), np.abs(gw - rw).max()
    return gid, gw


ROUTE_CASES = [
    # T, E, k, score, bias, G, Gk, group score, renorm, scale, type
    (1, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5, FP), (3000, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5, FP),
    (513, 256, 8, "sigmoid", False, 8, 4, "top2", True, 2.5, FP), (300, 160, 6, "softmax", False, 8, 3, "max", False, 16.0, BF),
    (700, 256, 8, "softmax", True, 1, 1, "top2", True, 1.0, FP), (100, 1024, 32, "sigmoid", True, 16, 5, "top2", True, 1.0, FP),
    (200, 1020, 7, "softmax", True, 5, 2, "top2", True, 1.0, FP), (64, 1020, 9, "sigmoid", True, 17, 3, "max", False, 1.0, HF),
    (33, 37, 5, "sigmoid", True, 1, 1, "top2", True, 1.0, FP), (9, 1, 1, "sigmoid", True, 1, 1, "top2", True, 1.0, FP),
    (9, 32, 4, "softmax", True, 32, 7, "top2", True, 1.0, FP), (50, 12, 3, "sigmoid", False, 3, 1, "max", True, 1.0, BF),
    (50, 64, 16, "softmax", True, 4, 4, "top2", False, 0.5, HF), (40, 8, 8, "sigmoid", True, 2, 2, "top2", True, 1.0, FP),
    (128, 384, 8, "sigmoid", True, 1, 1, "top2", True, 2.5, BF),
]


@pytest.mark.parametrize("T,E,k,score,bias,G,Gk,gscore,renorm,scale,dt", ROUTE_CASES)
def test_route(moe, T, E, k, score, bias, G, Gk, gscore, renorm, scale, dt):
    logits = randn(T, E, seed=T + E, dtype=dt, scale=1.5)
    b = randn(E, seed=E, scale=0.05 if score == "sigmoid" else 0.3 / E) if bias else None
    check_route(moe, logits, k, score=score, bias=b, G=G, Gk=Gk, group_score=gscore, renorm=renorm, scale=scale)


def test_route_equals_the_softmax_router(moe):
    """Softmax without bias and groups is route_topk."""
    logits = randn(777, 256, seed=3)
    a = moe.route_topk(logits, 8)
    b = moe.route_scored(logits, 8, score="softmax")
    assert torch.equal(a[0], b[0])
    check(b[1], a[1], 256 * U, "weights")


def test_route_ties_go_to_the_lower_index(moe):
    E = 256
    logits = (randn(400, E, seed=4) * 2).round() / 2                # many equal logits
    logits[0] = 0.25
    for bias in (None, torch.zeros(E, device="cuda"), (randn(E, seed=5) * 2).round() * 0.0625):
        for G, Gk in ((1, 1), (8, 4)):
            for score in ("sigmoid", "softmax"):
                gid, _ = check_route(moe, logits, 8, score=score, bias=bias, G=G, Gk=Gk)
                if bias is None:
                    assert gid[0].tolist() == list(range(8))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_of_nearly_equal_scores(moe, score):
    """Pairs whose choice values differ by less than fp32 can tell: biases chosen
    so that s_a + b_a and s_b + b_b agree to fp32 rounding."""
    T, E = 500, 64
    logits = randn(T, E, seed=6)
    logits[1:] = logits[0]                                          # the same near ties in every token ...
    z = logits[0].double()
    s = 1 / (1 + torch.exp(-z)) if score == "sigmoid" else torch.softmax(z, 0)
    bias = torch.zeros(E, dtype=torch.float64, device="cuda")
    bias[1::2] = s[0::2] - s[1::2]                                  # expert 2i + 1 as good as 2i
    bias = bias.float()
    logits += torch.linspace(0, 1e-4, T, device="cuda")[:, None]    # ... a little apart
    check_route(moe, logits, 9, score=score, bias=bias)
    check_route(moe, logits, 9, score=score, bias=bias, G=8, Gk=3)
    groups = logits.clone()
    groups[:, 32:] = groups[:, :32]                                 # equal groups
    check_route(moe, groups, 9, score=score, bias=torch.cat([bias[:32], bias[:32]]), G=2, Gk=1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,Gk", [(1, 1), (8, 3), (4, 2)])
def test_route_when_all_scores_are_nearly_equal(moe, score, G, Gk):
    """More values within fp32's error of one another than are collected at a time."""
    T, E = 60, 256
    logits = randn(T, E, seed=16)
    logits[1:] = logits[0]
    z = logits[0].double()
    s = 1 / (1 + torch.exp(-z)) if score == "sigmoid" else torch.softmax(z, 0)
    bias = (s.max() - s).float()                                    # every choice value is s.max() to fp32
    logits += torch.linspace(0, 1e-6, T, device="cuda")[:, None]
    for k in (1, 8, 32):
        check_route(moe, logits, k, score=score, bias=bias, G=G, Gk=Gk)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [16, 31, 32])
def test_route_of_many_nearly_equal_pairs(moe, score, k):
    """Many experts chosen of many: every value has another one next to it, nearer than fp32's error."""
    T, E = 40, 1024
    logits = randn(T, E, seed=k)
    logits[1:] = logits[0]
    z = logits[0].double()
    s = 1 / (1 + torch.exp(-z)) if score == "sigmoid" else torch.softmax(z, 0)
    bias = randn(E, seed=k + 1, scale=0.05)
    bias[512:] = (s[:512] + bias[:512].double() - s[512:]).float()
    logits += torch.linspace(0, 1e-6, T, device="cuda")[:, None]
    check_route(moe, logits, k, score=score, bias=bias)
    check_route(moe, logits, k, score=score, bias=bias, G=4, Gk=2)


@pytest.mark.parametrize("k", [1, 7, 15, 16, 24, 31, 32])
def test_route_topk_sizes(moe, k):
    """The bound below the chosen ones comes from the lanes' best or second best values, by k and the lanes in play."""
    for E, G, Gk in ((1024, 1, 1), (256, 8, 8), (256, 8, 2), (512, 16, 3), (64, 1, 1), (96, 3, 1)):
        if k <= Gk * (E // G):
            check_route(moe, randn(90, E, seed=k + E), k, bias=randn(E, seed=E, scale=0.05), G=G, Gk=Gk)
            check_route(moe, randn(90, E, seed=k + E + 1, dtype=BF), k, score="softmax", G=G, Gk=Gk, group_score="max")


def test_route_weights_of_experts_far_below_the_largest(moe):
    """Chosen by bias: softmax scores around and below fp32's smallest, divided by their sum."""
    logits = randn(64, 64, seed=21, scale=3.0) - torch.linspace(0, 300, 64, device="cuda")[:, None]
    logits[:, 5] = 20.0
    bias = torch.zeros(64, device="cuda")
    bias[16:32] = 4.0                                               # the group without the largest logit
    for k in (1, 6, 16):
        _, w = check_route(moe, logits, k, score="softmax", bias=bias, G=4, Gk=1)
        assert np.abs(w.sum(axis=1) - 1).max() < 1e-5
    z = torch.full((8, 16), -88.5, device="cuda") + randn(8, 16, seed=22, scale=0.1)
    _, w = moe.route_scored(z, 4)                                   # sigmoids below 2^-126
    assert bool(torch.isfinite(w).all()) and bool(((w.sum(dim=1) - 1).abs() < 1e-2).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_masked_experts(moe, score):
    inf = float("inf")
    logits = randn(12, 32, seed=7)
    logits[0] = -inf                                                # nothing left
    logits[1, 1:] = -inf                                            # one expert left
    logits[2, 4] = float("nan")
    logits[3, 5] = inf
    logits[4, 5:8] = inf
    logits[5] = float("nan")
    logits[6, :28] = -inf
    logits[7] = torch.finfo(FP).min                                 # a mask of the type's lowest value
    logits[8, 2:] = torch.finfo(FP).min
    bias = randn(32, seed=8, scale=0.01)
    for b in (None, bias):
        for G, Gk in ((1, 1), (4, 2)):
            gid, gw = check_route(moe, logits, 4, score=score, bias=b, G=G, Gk=Gk)
            assert not gw[0].any() and not gw[5].any()
            if b is None:
                assert gid[0].tolist() == [0, 1, 2, 3]


def test_route_strided_rows_and_empty(moe):
    wide = randn(40, 300, seed=9)
    a = moe.route_scored(wide[:, 3:259], 8, groups=8, topk_groups=4)
    b = moe.route_scored(wide[:, 3:259].contiguous(), 8, groups=8, topk_groups=4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ids, w = moe.route_scored(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


# ---------------------------------------------------------------- linear


def codes(*shape, seed=0, lo=-128):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(lo, 128, shape, generator=g, device="cuda", dtype=torch.int16).to(I8)


def check_linear(moe, T, K, N, dt=BF, bias=False, addend=False, seed=0, xq=None, wq=None, extra=0.0, **kw):
    xq = codes(T, K, seed=seed) if xq is None else xq
    wq = codes(N, K, seed=seed + 1) if wq is None else wq
    xs, ws = randn(T, seed=seed + 2).abs() * 1e-2 + 1e-3, randn(N, seed=seed + 3).abs() * 1e-2 + 1e-3
    b = randn(N, seed=seed + 4) if bias else None
    a = randn(T, N, seed=seed + 5, dtype=dt) if addend else None
    out = moe.linear_q8(xq, xs, wq, ws, bias=b, addend=a, dtype=dt, **kw)
    p = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
    ref, mag = p.clone(), p.abs()
    for v in (b, a):
        if v is not None:
            ref = ref + v.double()
            mag = mag + v.double().abs()
    check(out, ref, half_step(dt), f"linear {T}x{K}x{N}", extra=(5 * U + extra) * mag, floor=2.0 ** -25 if dt == HF else 0.0)
    return out


LINEAR_CASES = [
    (1, 16, 1, FP), (1, 4096, 4096, BF), (4, 2048, 4096, BF), (5, 4080, 33, FP), (8, 48, 100, HF), (9, 1024, 17, FP),
    (16, 4096, 256, BF), (17, 528, 40, FP), (31, 64, 1000, FP), (32, 4096, 640, BF),
    (33, 4096, 512, FP), (64, 16, 1, FP), (64, 4096, 4096, BF), (65, 1040, 129, FP), (77, 2048, 1000, BF),
    (128, 4096, 128, HF), (129, 80, 257, FP), (200, 4096, 1408, FP), (255, 2064, 300, FP), (256, 4096, 4096, BF),
    (257, 1024, 1023, FP), (512, 8192, 640, FP), (1000, 4096, 2050, BF), (2048, 512, 4096, FP), (3001, 1008, 777, FP),
    # few tokens, many blocks; sums of more than 1024 products per warp
    (4, 256, 5003, BF), (13, 512, 6000, FP), (30, 128, 8000, HF), (3, 65536, 40, FP), (20, 16384, 16, FP),
    # more than 32 tokens with few channels, in groups of 32 and of fewer; the last group with one token
    (33, 128, 17, FP), (40, 512, 512, HF), (97, 2048, 1000, BF), (600, 1024, 256, FP), (1000, 128, 64, BF),
    # and with many channels: small tiles of tokens, an odd number of channels
    (40, 256, 8192, BF), (100, 512, 4096, FP), (70, 2048, 8192, HF), (300, 16, 5003, FP), (129, 80, 6001, FP),
    (1000, 4096, 1025, FP),
    # few tokens, long sums and many channels
    (33, 4096, 4099, FP), (90, 8192, 2048, HF), (48, 4112, 5001, FP), (64, 4000, 16000, BF), (100, 16384, 1600, FP),
    # tokens on the M side, with ragged tiles of them
    (3001, 1008, 784, BF), (2500, 256, 1040, HF), (4100, 128, 512, BF), (5000, 1040, 4096, BF), (1700, 2048, 1408, FP),
]


@pytest.mark.parametrize("T,K,N,dt", LINEAR_CASES)
def test_linear(moe, T, K, N, dt):
    check_linear(moe, T, K, N, dt, seed=T + K)
    check_linear(moe, T, K, N, dt, bias=True, addend=True, seed=T + K + 7)


@pytest.mark.parametrize("T", [4, 40, 300, 3000])
def test_linear_extreme_codes(moe, T):
    """All codes -128 or 127: sums of K * 2^14 leave the range in which fp32 sums
    are exact; small batches add integers, larger ones stay within 2^-23 per 16 k."""
    K, N = 4096, 256
    for a, b in ((-128, -128), (127, 127), (-128, 127)):
        xq = torch.full((T, K), a, dtype=I8, device="cuda")
        wq = torch.full((N, K), b, dtype=I8, device="cuda")
        check_linear(moe, T, K, N, FP, xq=xq, wq=wq, extra=0.0 if T <= 32 else K / 16 * 2.0 ** -23)
    K = 1024                                                        # always below 2^24
    check_linear(moe, T, K, N, FP, xq=torch.full((T, K), -128, dtype=I8, device="cuda"),
                 wq=torch.full((N, K), 127, dtype=I8, device="cuda"))


def test_linear_is_reproducible_and_adds_in_place(moe):
    for T in (3, 100, 700):
        xq, wq = codes(T, 2048, seed=1), codes(512, 2048, seed=2)
        xs, ws = randn(T, seed=3).abs(), randn(512, seed=4).abs()
        a = randn(T, 512, seed=5, dtype=BF)
        first = moe.linear_q8(xq, xs, wq, ws, addend=a)
        for _ in range(3):
            assert torch.equal(first, moe.linear_q8(xq, xs, wq, ws, addend=a))
        b = a.clone()
        assert moe.linear_q8(xq, xs, wq, ws, addend=b, out=b) is b and torch.equal(first, b)


def test_linear_workspace_and_status(moe):
    T, K, N = 300, 1024, 512
    n = moe.linear_q8_workspace_size(T, K, N)
    ws = torch.full((n + 256,), 0x5a, dtype=torch.uint8, device="cuda")   # nothing needs to be cleared before
    a = check_linear(moe, T, K, N, workspace=ws[:n], seed=1)
    assert bool((ws[n:] == 0x5a).all())
    assert moe.read_status(ws) == moe.OK
    b = check_linear(moe, T, K, N, workspace=ws[:n], seed=1)
    assert torch.equal(a, b)
    with pytest.raises(moe.Wna16Error):
        check_linear(moe, T, K, N, workspace=ws[:n - 256], seed=1)


def test_debug_build_matches_release(moe):
    """The bounds-checked build gives the same bits."""
    from wna16_grouped_gemm_gb300 import binding, block, build
    build.build(debug=True)
    saved = block._load()
    outs = []
    try:
        for lib in (saved, block.declare(binding.load_debug_library())):
            block._lib = lib
            outs.append([check_linear(moe, T, K, N, FP, seed=T) for T, K, N in ((7, 528, 50), (70, 1040, 130), (600, 2048, 1024))])
    finally:
        block._lib = saved
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- streams, graphs, the block


def _block_inputs(T, dt=BF, E=8, K=512, N=256, Ns=384, seed=0):
    import synth
    import wna16_grouped_gemm_gb300 as moe
    wl = synth.Workload("blk", T=T, K=K, N=N, E=E, topk=2, bits=4, g13=128, g2=128, scale_lo=0.001, scale_hi=0.005)
    w13p, w13s, w2p, w2s = (torch.from_numpy(a).cuda() for a in synth.make_weights(wl, seed))
    s13, s13s = moe.quantize_q8(randn(2 * Ns, K, seed=1, scale=K ** -0.5))
    s2, s2s = moe.quantize_q8(randn(K, Ns, seed=2, scale=Ns ** -0.5))
    w = moe.MoEBlockWeights(norm=(1 + 0.2 * randn(K, seed=3)).to(dt), gate=randn(E, K, seed=4, dtype=dt, scale=2 * K ** -0.5),
                            gate_bias=randn(E, seed=5, scale=0.05), w13_packed=w13p, w13_scales=w13s, w2_packed=w2p,
                            w2_scales=w2s, shared_w13=s13, shared_w13_scales=s13s, shared_w2=s2, shared_w2_scales=s2s)
    kw = dict(topk=2, bits=4, group_size=128, groups=4, topk_groups=2, scale=1.5)
    return randn(T, K, seed=6, dtype=dt), randn(T, K, seed=7, dtype=dt), w, kw


@pytest.mark.parametrize("T", [1, 5, 100, 700])
def test_moe_block(moe, oracle, T):
    """The block's output against its parts in 64 bits on the host: the routed
    experts by the oracle, the shared expert by plain products of the values
    that the 8-bit rows stand for.  Tolerance: the framework's relative L2 of
    1e-3 for the routed part, and of the shared part a bf16 rounding (2^-9)
    before the second quantisation, whose rounding of at most half a step of
    m / 127 makes a relative error of (1/127) / sqrt(12) * (m / rms) < 1.5e-2 of
    h; the sum of both, rounded to bf16."""
    from tests import gpu_util as gu
    x, r, w, kw = _block_inputs(T)
    out, res = moe.moe_block(x, r, w, **kw)
    h, y = norm_ref(x, w.norm, r, 1e-6)
    check(res, h, half_step(BF) + 2 * U, "residual")
    q, s, _, normed = moe.add_rmsnorm_q8(x, w.norm, r, want_norm=True)
    ids, wts = moe.route_scored(normed @ w.gate.t(), 2, bias=w.gate_bias, groups=4, topk_groups=2, scale=1.5)
    routed = oracle.forward(gu.host_bits(normed), ids.cpu().numpy(), wts.cpu().numpy(), w.w13_packed.cpu().numpy(),
                            w.w13_scales.cpu().numpy(), w.w2_packed.cpu().numpy(), w.w2_scales.cpu().numpy(), bits=4,
                            group_size=128, group_size_w2=128, swiglu_limit=7.0)
    gate, up = ((q.double() * s.double()) @ (w.shared_w13.double() * w.shared_w13_scales.double()).t()).chunk(2, dim=1)
    gate, up = gate.clamp(max=7.0), up.clamp(-7.0, 7.0)
    shared = (gate / (1 + torch.exp(-gate)) * up) @ (w.shared_w2.double() * w.shared_w2_scales.double()).t()
    ref = torch.from_numpy(gu.bf16_bits_to_f64(routed)).cuda()
    tol = 1.5e-2 * float(shared.norm()) + (1e-3 + 2.0 ** -8) * float(ref.norm() + shared.norm())
    assert float((out.double() - ref - shared).norm()) <= tol


def test_other_stream_and_graph(moe):
    """The block on a side stream and replayed from a graph with new inputs gives the bits of the eager call."""
    x, r, w, kw = _block_inputs(48)
    out, res = moe.moe_block(x, r, w, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, r2 = moe.moe_block(x, r, w, **kw)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(res, r2)
    q = moe.quantize_q8(x, stream=side)
    side.synchronize()
    assert torch.equal(q[0], moe.quantize_q8(x)[0])
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


def test_wrappers_refuse(moe):
    x = randn(4, 64, dtype=BF)
    w = torch.ones(64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        moe.add_rmsnorm_q8(x, w, x[:3])
    with pytest.raises(TypeError):
        moe.add_rmsnorm_q8(x, w, x.half())
    with pytest.raises(TypeError):
        moe.add_rmsnorm_q8(x, w.half())
    with pytest.raises(ValueError):
        moe.add_rmsnorm_q8(x.t(), w)                                # rows not contiguous
    with pytest.raises(moe.Wna16Error):
        moe.quantize_q8(x[:1].expand(4, 64))                        # rows on top of each other
    with pytest.raises(TypeError):
        moe.quantize_q8(x, q_dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.quantize_q8(x, q=torch.empty(4, 63, dtype=I8, device="cuda"))
    with pytest.raises(ValueError):
        moe.swiglu_q8(x[:, :63])
    with pytest.raises(ValueError):
        moe.route_scored(x, 2, score="tanh")
    with pytest.raises(moe.Wna16Error):
        moe.route_scored(x, 2, groups=5)
    with pytest.raises(moe.Wna16Error):
        moe.route_scored(x, 40)
    q, s = moe.quantize_q8(x)
    with pytest.raises(ValueError):
        moe.linear_q8(q, s, q[:, :32].contiguous(), s)
    with pytest.raises(ValueError):
        moe.linear_q8(q, s[:2], q, s)
    with pytest.raises(moe.Wna16Error):
        moe.linear_q8(q[:, :8].contiguous(), s, q[:, :8].contiguous(), s)
    with pytest.raises(ValueError):
        moe.dequantize_q8(q, torch.ones(4, 5, device="cuda"))
