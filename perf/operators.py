"""The operators around the routed experts, as workloads that can be timed and compared.

A transformer layer with routed experts reaches them through four operators:

  norm    residual addition, root-mean-square norm, and the normed rows in 8 bits with their scales
          (the routed experts and the router read the norm's 16-bit output, the shared expert the 8-bit one)
  route   expert scores (sigmoid or softmax), a selection bias, groups of experts, top-k, weights
  linear  the shared expert's products: 8-bit integers, one scale per token and one per output channel
  swiglu  the clamped SwiGLU between its two products, in 8 bits with scales for the second one

`run` computes one pass of one of them: in elementary torch operations, or with `own` set through this
repository's package.  8-bit outputs are returned as the values that they stand for (code times scale).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
QMAX = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-6
LIMIT = 7.0
#: rows whose largest magnitude is below this are stored as zeros with scale 0
TINY = 2.0 ** -100
BIGGEST = 8192 * 4096 * 4096


def listed():
    return [
        # one decode step of four sequences at the framework's hidden size: a launch's latency
        {"name": "norm decode", "op": "norm", "T": 4, "K": 4096, "dtype": "bf16", "q": "int8", "group": 0, "residual": True, "normed": True},
        # a long prefill: every byte of the residual stream passes once
        {"name": "norm prefill", "op": "norm", "T": 8192, "K": 4096, "dtype": "bf16", "q": "int8", "group": 0, "residual": True, "normed": True},
        # activations for a block-scaled 8-bit float layer: scales per 128 elements, an odd token count
        {"name": "norm e4m3 g128", "op": "norm", "T": 2047, "K": 5120, "dtype": "fp16", "q": "e4m3", "group": 128, "residual": True, "normed": False},
        # the shared expert's activation in the same decode step
        {"name": "swiglu decode", "op": "swiglu", "T": 4, "N": 2048, "dtype": "bf16", "q": "int8", "group": 0},
        # and in the long prefill
        {"name": "swiglu prefill", "op": "swiglu", "T": 8192, "N": 2048, "dtype": "bf16", "q": "int8", "group": 0},
        # 256 experts in 8 groups, 4 groups and 8 experts kept: one decode step
        {"name": "route decode", "op": "route", "T": 4, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "G": 8, "Gk": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # the same router over a long prefill
        {"name": "route prefill", "op": "route", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "G": 8, "Gk": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # softmax scores, groups by their best expert, group sizes that are no power of two, 16-bit logits
        {"name": "route softmax 160", "op": "route", "T": 2047, "E": 160, "k": 6, "score": "softmax", "bias": False, "G": 8, "Gk": 3, "group_score": "max", "renorm": False, "scale": 16.0, "dtype": "bf16"},
        # the shared expert's gate/up product in a decode step: the weights' bytes
        {"name": "linear decode", "op": "linear", "T": 4, "K": 4096, "N": 4096, "dtype": "bf16"},
        # a ragged batch against a small odd layer
        {"name": "linear ragged", "op": "linear", "T": 77, "K": 2048, "N": 1000, "dtype": "bf16"},
        # a prefill chunk, and a long prefill: the tensor cores
        {"name": "linear chunk", "op": "linear", "T": 2048, "K": 4096, "N": 4096, "dtype": "bf16"},
        {"name": "linear prefill", "op": "linear", "T": 8192, "K": 4096, "N": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "route", "linear"])
    T = _log(rng, 1, 8192)
    if op == "norm":
        group = rng.choice([0, 0, 32, 64, 128])
        K = rng.choice([128, 8]) * rng.randint(2, 40) if group == 0 else 128 * rng.randint(2, 40)
        if group == 0 and rng.random() < 0.25:
            K += rng.choice([1, 3, 7])
        return {"op": op, "T": min(T, 8192 * 4096 // K), "K": K, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "q": rng.choice(["int8", "e4m3"]), "group": group,
                "residual": rng.random() < 0.75, "normed": rng.random() < 0.5}
    if op == "swiglu":
        group = rng.choice([0, 0, 128])
        N = 128 * rng.randint(1, 32) if group else 8 * rng.randint(8, 512)
        return {"op": op, "T": T, "N": N, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "q": rng.choice(["int8", "e4m3"]), "group": group}
    if op == "route":
        G = rng.choice([1, 1, 4, 8, 16])
        E = G * rng.randint(2, 512 // G)
        Gk = rng.randint(1, G)
        k = rng.randint(1, min(16, Gk * (E // G)))
        score = rng.choice(["sigmoid", "softmax"])
        return {"op": op, "T": T, "E": E, "k": k, "score": score, "bias": rng.random() < 0.5, "G": G, "Gk": Gk, "group_score": rng.choice(["top2", "max"]),
                "renorm": rng.random() < 0.75, "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["fp32", "fp32", "bf16"])}
    K = 16 * rng.randint(8, 256)
    N = rng.choice([rng.randint(16, 300), 8 * rng.randint(16, 512), 128 * rng.randint(4, 64)])
    return {"op": op, "T": min(T, BIGGEST // (K * N)), "K": K, "N": N, "dtype": rng.choice(["bf16", "bf16", "fp16"])}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    u = lambda lo, hi, *s: lo + (hi - lo) * torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": case, "buf": {}}
    dt = DTYPES[case["dtype"]]
    T = case["T"]
    if case["op"] == "norm":
        K = case["K"]
        channel = torch.exp(0.5 * n(K))  # a residual stream's channels have sizes of their own
        s["x"] = (n(T, K) * 0.5).to(dt)
        s["residual"] = (n(T, K) * channel).to(dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * n(K)).to(dt)
    elif case["op"] == "swiglu":
        s["gu"] = (n(T, 2 * case["N"]) * 2.0).to(dt)  # some gates and ups pass the limit
    elif case["op"] == "route":
        E = case["E"]
        s["logits"] = (n(T, E) + 0.5 * n(E)).to(dt)  # some experts are more popular
        s["bias"] = n(E) * (0.05 if case["score"] == "sigmoid" else 0.5 / E) if case["bias"] else None
    else:
        K, N = case["K"], case["N"]
        s["xq"] = (n(T, K) * 32).round().clamp(-127, 127).to(torch.int8)
        s["wq"] = (n(N, K) * 32).round().clamp(-127, 127).to(torch.int8)
        s["xs"], s["ws"] = u(0.01, 0.05, T), u(0.0005, 0.002, N)
    s["buf"] = _buffers(case)
    return s


def _buffers(case):
    """The outputs that a program keeps between its steps."""
    e = lambda dt, *s: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    T, dt = case["T"], DTYPES[case["dtype"]]
    if case["op"] in ("norm", "swiglu"):
        K = case["K"] if case["op"] == "norm" else case["N"]
        b = {"q": e(torch.int8 if case["q"] == "int8" else torch.float8_e4m3fn, T, K), "scales": e(torch.float32, T, K // case["group"] if case["group"] else 1), "values": e(dt, T, K)}
        if case.get("residual"):
            b["residual_out"] = e(dt, T, K)
        if case.get("normed"):
            b["norm_out"] = e(dt, T, K)
        return b
    if case["op"] == "route":
        return {"ids": e(torch.int32, T, case["k"]), "weights": e(torch.float32, T, case["k"])}
    return {"out": e(dt, T, case["N"])}


# ---------------------------------------------------------------- one pass


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import wna16_grouped_gemm_gb300 as moe
    c, b = s["case"], s["buf"]
    if c["op"] == "norm":
        q, scales, res, normed = moe.add_rmsnorm_q8(s["x"], s["weight"], s["residual"], eps=EPS, group_size=c["group"], q=b["q"], scales=b["scales"],
                                                    residual_out=b.get("residual_out"), norm_out=b.get("norm_out"))
        return {"residual": res, "normed": normed, "scales": scales, "values": moe.dequantize_q8(q, scales, out=b["values"])}
    if c["op"] == "swiglu":
        q, scales = moe.swiglu_q8(s["gu"], swiglu_limit=LIMIT, group_size=c["group"], q=b["q"], scales=b["scales"])
        return {"scales": scales, "values": moe.dequantize_q8(q, scales, out=b["values"])}
    if c["op"] == "route":
        ids, weights = moe.route_scored(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["G"], topk_groups=c["Gk"], group_score=c["group_score"],
                                        renormalize=c["renorm"], scale=c["scale"], ids=b["ids"], weights=b["weights"])
        return {"ids": ids, "weights": weights}
    return {"out": moe.linear_q8(s["xq"], s["xs"], s["wq"], s["ws"], out=b["out"])}


def _quantized(y, q, group, dt):
    """Scales and values of fp32 rows y held in 8 bits."""
    T, K = y.shape
    y = y.view(T, -1, group or K)
    amax = y.abs().amax(dim=2, keepdim=True)
    scale = torch.where(amax < TINY, 0.0, amax / QMAX[q])
    r = torch.where(scale == 0, 0.0, y / scale)
    r = r.round() if q == "int8" else r.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    return scale.view(T, -1), (r * scale).view(T, K).to(dt)


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        scales, values = _quantized(y, c["q"], c["group"], dt)
        return {"residual": h.to(dt) if s["residual"] is not None else None, "normed": y.to(dt) if c["normed"] else None, "scales": scales, "values": values}
    if c["op"] == "swiglu":
        g, up = s["gu"].float().split(c["N"], dim=1)
        g, up = g.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)
        scales, values = _quantized(g / (1 + torch.exp(-g)) * up, c["q"], c["group"], dt)
        return {"scales": scales, "values": values}
    if c["op"] == "route":
        # the order of nearly equal scores is that of 64-bit scores
        T, E, G = c["T"], c["E"], c["G"]
        z = s["logits"].double()
        if c["score"] == "sigmoid":
            score = 1 / (1 + torch.exp(-z))
        else:
            ex = torch.exp(z - z.amax(dim=1, keepdim=True))
            score = ex / ex.sum(dim=1, keepdim=True)
        choice = score if s["bias"] is None else score + s["bias"].double()
        if G > 1:
            grouped = choice.view(T, G, E // G)
            best = grouped.sort(dim=2, descending=True).values
            best = best[:, :, 0] if c["group_score"] == "max" else best[:, :, :2].sum(dim=2)
            kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["Gk"]]
            keep = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
            choice = torch.where(keep.unsqueeze(2), grouped, -math.inf).view(T, E)
        ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
        w = score.gather(1, ids)
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        return {"ids": ids.to(torch.int32), "weights": (w * c["scale"]).float()}
    acc = s["xq"].float() @ s["wq"].float().t()
    return {"out": (acc * s["xs"][:, None] * s["ws"][None, :]).to(dt)}


# ---------------------------------------------------------------- cost and definition


def work(case):
    T, c = case["T"], case
    b = 4 if c["dtype"] == "fp32" else 2
    if c["op"] in ("norm", "swiglu"):
        K = c["K"] if c["op"] == "norm" else c["N"]
        scales = 4 * T * (K // c["group"] if c["group"] else 1)
        out = T * K * (1 + b) + scales  # the codes and the values that they stand for
        if c["op"] == "swiglu":
            return {"bytes": 2 * T * K * b + out, "flops": 12 * T * K}
        return {"bytes": T * K * b * (1 + 2 * c["residual"] + c["normed"]) + K * b + out, "flops": 8 * T * K}
    if c["op"] == "route":
        return {"bytes": T * c["E"] * b + 4 * c["E"] * c["bias"] + 8 * T * c["k"], "flops": T * c["E"] * 8}
    K, N = c["K"], c["N"]
    return {"bytes": T * K + N * K + 4 * (T + N) + T * N * b, "flops": 2 * T * N * K}


def _held(y, q, group):
    """64-bit scales and values of y [T, K] held in 8 bits, by the numbers that a format has."""
    T, K = y.shape
    y = y.reshape(T, K // (group or K), group or K)
    m = np.abs(y).max(axis=2, keepdims=True)
    scale = np.where(m < TINY, 0.0, m / QMAX[q])
    a = y / np.where(scale == 0, 1.0, scale)
    if q == "e4m3":  # 3 bits behind the first, the smallest step 2^-9
        step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(a), 2.0 ** -12))), -6) - 3)
        a = np.rint(a / step) * step
    else:
        a = np.rint(a)
    return scale.reshape(T, -1), (a * scale).reshape(T, K)


def exact(case, seed):
    s = prepare(case, seed)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    c = case
    if c["op"] == "norm":
        h = host(s["x"])
        if s["residual"] is not None:
            h += host(s["residual"])
        y = h / np.sqrt(np.einsum("tk,tk->t", h, h)[:, None] / c["K"] + EPS)
        y *= host(s["weight"])
        scales, values = _held(y, c["q"], c["group"])
        return {"residual": h if s["residual"] is not None else None, "normed": y if c["normed"] else None, "scales": scales, "values": values}
    if c["op"] == "swiglu":
        gu = host(s["gu"])
        g, up = np.minimum(gu[:, :c["N"]], LIMIT), np.clip(gu[:, c["N"]:], -LIMIT, LIMIT)
        scales, values = _held(g * 0.5 * (1 + np.tanh(g / 2)) * up, c["q"], c["group"])
        return {"scales": scales, "values": values}
    if c["op"] == "route":
        z = host(s["logits"])
        p = 0.5 * (1 + np.tanh(z / 2)) if c["score"] == "sigmoid" else np.exp(z - np.log(np.exp(z).sum(axis=1, keepdims=True)))
        v = p + (0 if s["bias"] is None else host(s["bias"]))
        T, E = v.shape
        if c["G"] > 1:
            of = v.reshape(T, c["G"], -1)
            top = np.partition(of, of.shape[2] - min(2, of.shape[2]), axis=2)[:, :, -2:]
            rank = top.max(axis=2) if c["group_score"] == "max" else top.sum(axis=2)
            out = np.argsort(np.argsort(-rank, axis=1, kind="stable"), axis=1) >= c["Gk"]
            v = np.where(np.repeat(out, E // c["G"], axis=1), -np.inf, v)
        ids = np.argsort(-v, axis=1, kind="stable")[:, :c["k"]]
        w = np.take_along_axis(p, ids, axis=1)
        return {"ids": None, "weights": w / (w.sum(axis=1, keepdims=True) if c["renorm"] else 1.0) * c["scale"]}
    xq, wq = s["xq"].double(), s["wq"].double()
    out = torch.empty(c["T"], c["N"], dtype=torch.float64, device=xq.device)
    for at in range(0, c["T"], 1024):
        out[at:at + 1024] = xq[at:at + 1024] @ wq.t()
    return {"out": out.cpu().numpy() * host(s["xs"])[:, None] * host(s["ws"])[None, :]}
