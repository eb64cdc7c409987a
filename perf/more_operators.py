"""Routed experts in 8-bit floats, as workloads that can be timed and compared.

Experts whose weights are e4m3 codes with one scale per 128 x 128 block (as checkpoints in 8-bit floats
have them) take rows in e4m3 with one scale per 128 values.  A layer of them is:

  sort     tokens copied to rows in the order of their experts (16-bit rows, or 8-bit ones with their scales)
  experts  the products of each expert with its rows
  unsort   every token's rows back, weighted and added up; and the gradient of that
  linear   the same product with one weight for all rows (a shared expert, a projection)
  blocks   weights to e4m3 with a scale per 128 x 128 block

`run` computes one pass of one of them: in elementary torch operations, or with `own` set through this
repository's package.  8-bit outputs are returned as the values that they stand for (code times scale).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
B = 128          # values per scale
QMAX = 448.0
#: blocks whose largest magnitude is below this are stored as zeros with scale 0
TINY = 2.0 ** -100
BIGGEST = 65536 * 4096 * 4096


def listed():
    return [
        # one decode step of four sequences, 8-bit rows straight from the norm: a launch's latency
        {"name": "sort decode", "op": "sort", "T": 4, "k": 8, "E": 256, "total": 256, "begin": 0, "zipf": False, "K": 4096, "dtype": "e4m3"},
        # a long prefill with 16-bit rows: every byte moves once in and eight times out
        {"name": "sort prefill", "op": "sort", "T": 8192, "k": 8, "E": 256, "total": 256, "begin": 0, "zipf": False, "K": 4096, "dtype": "bf16"},
        # its way back, with the routing weights
        {"name": "unsort prefill", "op": "unsort", "T": 8192, "k": 8, "E": 256, "total": 256, "begin": 0, "zipf": False, "K": 4096, "dtype": "bf16", "weights": True, "back": False},
        # the gradient of that for a training batch of one GPU's share of the experts: skewed, an odd token count, slots left out
        {"name": "unsort gradient", "op": "unsort", "T": 2047, "k": 8, "E": 128, "total": 256, "begin": 0, "zipf": True, "K": 4096, "dtype": "bf16", "weights": True, "back": True},
        # the shared expert's gate/up product in a decode step: the weights' bytes
        {"name": "linear decode", "op": "linear", "T": 4, "K": 4096, "N": 4096, "dtype": "bf16"},
        # a ragged batch against a small odd layer
        {"name": "linear ragged", "op": "linear", "T": 77, "K": 2048, "N": 1000, "dtype": "fp16"},
        # a long prefill: the tensor cores
        {"name": "linear prefill", "op": "linear", "T": 8192, "K": 4096, "N": 4096, "dtype": "bf16"},
        # the routed gate/up products of a decode step of four sequences: some 30 experts with a row or two
        {"name": "experts decode", "op": "experts", "T": 4, "k": 8, "E": 256, "zipf": False, "K": 4096, "N": 4096, "dtype": "bf16"},
        # the routed down products of a prefill chunk
        {"name": "experts chunk", "op": "experts", "T": 2048, "k": 8, "E": 256, "zipf": False, "K": 2048, "N": 4096, "dtype": "bf16"},
        # the routed gate/up products of a long prefill with skewed popularity: experts of thousands of rows and of a few
        {"name": "experts prefill", "op": "experts", "T": 8192, "k": 8, "E": 256, "zipf": True, "K": 4096, "N": 4096, "dtype": "bf16"},
        # a shared expert's weights, when a model is loaded
        {"name": "blocks layer", "op": "blocks", "E": 1, "N": 1000, "K": 2048, "dtype": "bf16"},
        # a stack of routed experts' weights, kept in 32 bits by a trainer
        {"name": "blocks experts", "op": "blocks", "E": 16, "N": 4096, "K": 4096, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "unsort", "linear", "experts", "blocks"])
    if op in ("sort", "unsort"):
        total = rng.choice([8, 60, 64, 160, 256, 512])
        E = rng.choice([total, total, total // 4, total // 2])
        c = {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "E": E, "total": total, "begin": E * rng.randint(0, total // E - 1),
             "zipf": rng.random() < 0.5, "K": B * rng.randint(2, 48)}
        if op == "sort":
            c["dtype"] = rng.choice(["bf16", "fp16", "fp32", "e4m3", "e4m3"])
        else:
            c |= {"dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "weights": rng.random() < 0.75, "back": rng.random() < 0.5}
        if c["dtype"] != "e4m3" and rng.random() < 0.25:
            c["K"] += rng.choice([1, 8, 100])
        c["T"] = min(c["T"], 8192 * 8 * 4096 * 2 // (c["k"] * c["K"] * max(2, SIZE[c["dtype"]])))
        return c
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    K = B * rng.randint(1, 48)
    N = rng.choice([rng.randint(16, 300), 8 * rng.randint(16, 768), 128 * rng.randint(4, 48)])
    if op == "linear":
        return {"op": op, "T": min(_log(rng, 1, 16384), BIGGEST // (K * N)), "K": K, "N": N, "dtype": dtype}
    if op == "experts":
        E = rng.choice([8, 16, 60, 128, 160, 256])
        k = rng.randint(1, 8)
        return {"op": op, "T": min(_log(rng, 1, 8192), BIGGEST // (k * K * N)), "k": k, "E": E, "zipf": rng.random() < 0.5, "K": K, "N": N, "dtype": dtype}
    return {"op": op, "E": rng.choice([1, 1, 3, 16]), "N": N, "K": K, "dtype": rng.choice(["bf16", "fp16", "fp32"])}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _popularity(n, zipf):
    """Shares of n experts (by rank, with zipf)."""
    p = [1.0 / (e + 1) if zipf else 1.0 for e in range(n)]
    return [v / sum(p) for v in p]


def _routing(case, g, n):
    """topk_ids int32 [T, k]: distinct experts of a token, by noise and popularity."""
    p = torch.tensor(_popularity(n, case["zipf"]), device="cuda").log()
    z = p[torch.randperm(n, generator=g, device="cuda")] + torch.randn(case["T"], n, generator=g, device="cuda")
    return z.topk(case["k"], dim=1).indices.to(torch.int32)


def _slots(ids, E, begin):
    """Of each slot the row that it has in the order of the experts, and the experts' first rows."""
    flat = ids.reshape(-1).long() - begin
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    ordered, order = key.sort(stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(order.numel(), device=order.device)
    inv = torch.where(key < E, inv, -1).to(torch.int32).view_as(ids)
    offsets = torch.searchsorted(ordered, torch.arange(E + 1, device=ids.device)).to(torch.int32)
    return order, ordered, inv, offsets


def _codes(g, *shape):
    """e4m3 codes as quantised rows have them: the largest of a block near 448."""
    return torch.randn(*shape, generator=g, device="cuda").mul_(120.0).clamp_(-QMAX, QMAX).to(torch.float8_e4m3fn)


def _weights(g, E, N, K):
    return _codes(g, E, N, K), (0.5 + torch.rand(E, -(-N // B), K // B, generator=g, device="cuda")) * 2e-4


def prepare(case, seed):
    g = _gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    z = lambda dt, *s: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    c, s, dt = case, {"case": case}, DTYPES[case["dtype"]]
    if c["op"] == "blocks":
        # channels have sizes of their own
        s["w"] = (n(c["E"], c["N"], c["K"]) * 0.02 * torch.exp(0.3 * n(c["E"], c["N"], 1))).to(dt)
        s["q"], s["scales"] = z(torch.float8_e4m3fn, c["E"], c["N"], c["K"]), z(torch.float32, c["E"], -(-c["N"] // B), c["K"] // B)
        s["values"] = z(torch.bfloat16, c["E"] * c["N"], c["K"])
        return s
    T, K = c["T"], c["K"]
    if c["op"] == "linear":
        w, ws = _weights(g, 1, c["N"], K)
        s["wq"], s["ws"] = w[0], ws[0]
        s["xq"], s["xs"] = _codes(g, T, K), torch.exp(0.3 * n(T, K // B)) * 0.005
        s["out"] = z(dt, T, c["N"])
        return s
    if c["op"] == "experts":
        ids = _routing(c, g, c["E"])
        s["offsets"] = _slots(ids, c["E"], 0)[3]
        s["wq"], s["ws"] = _weights(g, c["E"], c["N"], K)
        s["xq"], s["xs"] = _codes(g, T * c["k"], K), torch.exp(0.3 * n(T * c["k"], K // B)) * 0.005
        s["out"] = z(dt, T * c["k"], c["N"])
        return s
    ids = _routing(c, g, c["total"])
    R, E = T * c["k"], c["E"]
    if c["op"] == "sort":
        s["ids"] = ids
        s["offsets"], s["inv"], s["rows"] = z(torch.int32, E + 1), z(torch.int32, T, c["k"]), z(dt, R, K)
        if c["dtype"] == "e4m3":
            s["x"], s["xs"] = _codes(g, T, K), torch.exp(0.3 * n(T, K // B)) * 0.005
            s["row_scales"], s["values"] = z(torch.float32, R, K // B), z(torch.bfloat16, R, K)
        else:
            s["x"] = n(T, K).to(dt)
        return s
    s["inv"] = _slots(ids, E, c["begin"])[2]
    w = torch.rand(T, c["k"], generator=g, device="cuda") + 0.1
    s["weights"] = w / w.sum(dim=1, keepdim=True) if c["weights"] else None
    s["y"] = n(R, K).to(dt)
    if c["back"]:
        s["dout"], s["dy"], s["dweights"] = n(T, K).to(dt), z(dt, R, K), z(torch.float32, T, c["k"])
    else:
        s["out"] = z(dt, T, K)
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import wna16_grouped_gemm_gb300 as moe
    c = s["case"]
    if c["op"] == "sort":
        rows, scales, offsets, inv = moe.sort_tokens(s["x"], s["ids"], c["E"], scales=s.get("xs"), expert_begin=c["begin"], rows=s["rows"], row_scales=s.get("row_scales"),
                                                     offsets=s["offsets"], inv=s["inv"])
        if c["dtype"] != "e4m3":
            return {"rows": rows, "offsets": offsets, "inv": inv}
        return {"rows": moe.dequantize_q8(rows, scales, out=s["values"]), "scales": scales, "offsets": offsets, "inv": inv}
    if c["op"] == "unsort":
        if not c["back"]:
            return {"out": moe.unsort_tokens(s["y"], s["inv"], s["weights"], out=s["out"])}
        if s["weights"] is None:
            return {"dy": moe.unsort_tokens_grad(s["dout"], s["inv"], dy=s["dy"])[0]}
        dy, dweights = moe.unsort_tokens_grad(s["dout"], s["inv"], s["y"], s["weights"], dy=s["dy"], dweights=s["dweights"])
        return {"dy": dy, "dweights": dweights}
    if c["op"] == "linear":
        return {"out": moe.linear_f8(s["xq"], s["xs"], s["wq"], s["ws"], out=s["out"])}
    if c["op"] == "experts":
        return {"out": moe.grouped_linear_f8(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], out=s["out"])}
    q, scales = moe.quantize_blocks_f8(s["w"], q=s["q"], scales=s["scales"])
    rows = scales.repeat_interleave(B, dim=1)[:, :c["N"]].reshape(-1, c["K"] // B)
    return {"scales": scales, "values": moe.dequantize_q8(q.view(-1, c["K"]), rows, out=s["values"])}


def _values(q, scales):
    """fp32 values of e4m3 rows with a scale per 128."""
    return (q.float().view(q.shape[0], -1, B) * scales.unsqueeze(2)).view(q.shape)


def _block_values(q, scales):
    return _values(q, scales.repeat_interleave(B, dim=0)[:q.shape[0]])


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "sort":
        order, ordered, inv, offsets = _slots(s["ids"], c["E"], c["begin"])
        used = (ordered < c["E"]).unsqueeze(1)
        if c["dtype"] != "e4m3":
            return {"rows": torch.where(used, s["x"][order // c["k"]], 0), "offsets": offsets, "inv": inv}
        scales = torch.where(used, s["xs"][order // c["k"]], 0)
        rows = torch.where(used, _values(s["x"], s["xs"]).to(torch.bfloat16)[order // c["k"]], 0)
        return {"rows": rows, "scales": scales, "offsets": offsets, "inv": inv}
    if c["op"] == "unsort":
        used = s["inv"] >= 0
        at = s["inv"].long().clamp(min=0)
        w = used.float() if s["weights"] is None else torch.where(used, s["weights"], 0)
        if not c["back"]:
            return {"out": (s["y"].float()[at] * w.unsqueeze(2)).sum(dim=1).to(dt)}
        d = s["dout"].float()
        dy = torch.zeros_like(s["y"])
        dy[at[used]] = (d.unsqueeze(1) * w.unsqueeze(2)).to(dt)[used]
        if s["weights"] is None:
            return {"dy": dy}
        return {"dy": dy, "dweights": torch.where(used, (s["y"].float()[at] * d.unsqueeze(1)).sum(dim=2), 0)}
    if c["op"] == "linear":
        return {"out": (_values(s["xq"], s["xs"]) @ _block_values(s["wq"], s["ws"]).t()).to(dt)}
    if c["op"] == "experts":
        # experts have as many rows as the routing gives them: one product each, and the counts come to the host
        x, out = _values(s["xq"], s["xs"]), torch.zeros_like(s["out"])
        at = s["offsets"].tolist()
        for e in range(c["E"]):
            if at[e + 1] > at[e]:
                out[at[e]:at[e + 1]] = (x[at[e]:at[e + 1]] @ _block_values(s["wq"][e], s["ws"][e]).t()).to(dt)
        return {"out": out}
    E, N, K = s["w"].shape
    Nb = -(-N // B) * B
    w = torch.zeros(E, Nb, K, device="cuda")
    w[:, :N] = s["w"].float()
    w = w.view(E, Nb // B, B, K // B, B)
    amax = w.abs().amax(dim=(2, 4), keepdim=True)
    scales = torch.where(amax < TINY, 0.0, amax / QMAX)
    q = torch.where(scales == 0, 0.0, w / scales).clamp(-QMAX, QMAX).to(torch.float8_e4m3fn).float() * scales
    return {"scales": scales.view(E, Nb // B, K // B), "values": q.view(E, Nb, K)[:, :N].reshape(E * N, K).to(torch.bfloat16)}


# ---------------------------------------------------------------- cost and definition


def work(case):
    c, K, b = case, case["K"], SIZE[case["dtype"]]
    if c["op"] == "blocks":
        n = c["E"] * c["N"] * K
        # the codes and the values that they stand for
        return {"bytes": n * (b + 1 + 2) + 4 * c["E"] * -(-c["N"] // B) * (K // B), "flops": 3 * n}
    T = c["T"]
    if c["op"] == "linear":
        N = c["N"]
        return {"bytes": T * K + 4 * T * (K // B) + N * K + 4 * -(-N // B) * (K // B) + T * N * b, "flops": 2 * T * N * K}
    R = T * c["k"]
    if c["op"] == "experts":
        N = c["N"]
        active = sum(1 - (1 - p) ** R for p in _popularity(c["E"], c["zipf"]))  # experts with a row, on average
        return {"bytes": int(R * K + 4 * R * (K // B) + active * (N * K + 4 * -(-N // B) * (K // B)) + R * N * b), "flops": 2 * R * N * K}
    share = sum(_popularity(c["total"], False)[:c["E"]])  # of the slots that stay
    rows = int(R * share)
    if c["op"] == "sort":
        lists = 8 * R + 4 * (c["E"] + 1)
        if c["dtype"] == "e4m3":
            return {"bytes": T * (K + 4 * (K // B)) + rows * (K + 4 * (K // B) + 2 * K) + lists, "flops": rows * K}
        return {"bytes": (T + rows) * K * b + lists, "flops": 0}
    if not c["back"]:
        return {"bytes": (T + rows) * K * b + 8 * R, "flops": 2 * rows * K}
    return {"bytes": (T + rows * (2 if c["weights"] else 1)) * K * b + 12 * R, "flops": 3 * rows * K}


def _e4m3(a):
    """a (64-bit) to the nearest value that e4m3 has: 3 bits behind the first, the smallest step 2^-9."""
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(a), 2.0 ** -12))), -6) - 3)
    return np.rint(a / step) * step


def _product(xq, xs, wq, ws):
    """sum_b xs[t, b] ws[n / 128, b] sum_k x w, in 64 bits: scales taken out of each block of 128."""
    T, K = xq.shape
    w = wq.double() * ws.double().repeat_interleave(B, dim=0)[:wq.shape[0]].repeat_interleave(B, dim=1)
    out = torch.empty(T, wq.shape[0], dtype=torch.float64, device=xq.device)
    for at in range(0, T, 2048):
        out[at:at + 2048] = (xq[at:at + 2048].double() * xs[at:at + 2048].double().repeat_interleave(B, dim=1)) @ w.t()
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "linear":
        return {"out": _product(s["xq"], s["xs"], s["wq"], s["ws"]).cpu().numpy()}
    if c["op"] == "experts":
        first = s["offsets"].cpu().numpy()
        out = np.zeros(s["out"].shape)
        for e in np.flatnonzero(np.diff(first)):
            part = slice(int(first[e]), int(first[e + 1]))
            out[part] = _product(s["xq"][part], s["xs"][part], s["wq"][e], s["ws"][e]).cpu().numpy()
        return {"out": out}
    if c["op"] == "blocks":
        w = s["w"].double().cpu().numpy()
        scales, values = np.zeros(s["scales"].shape), np.empty(w.shape)
        for i in range(scales.shape[1]):
            rows = w[:, B * i:B * i + B].reshape(c["E"], -1, c["K"] // B, B)
            m = np.abs(rows).max(axis=(1, 3))
            scales[:, i] = np.where(m < TINY, 0.0, m / QMAX)
            by = scales[:, i][:, None, :, None]
            values[:, B * i:B * i + B] = (_e4m3(rows / np.where(by == 0, 1.0, by)) * by).reshape(c["E"], -1, c["K"])
        return {"scales": scales, "values": values.reshape(-1, c["K"])}
    T, k, K = c["T"], c["k"], c["K"]
    if c["op"] == "sort":
        ids = s["ids"].cpu().numpy().reshape(-1) - c["begin"]
        kept = np.flatnonzero((ids >= 0) & (ids < c["E"]))
        source = kept[np.argsort(ids[kept], kind="stable")] // k  # the token of each row
        x = s["x"].double().cpu().numpy()
        if c["dtype"] == "e4m3":
            sc = s["xs"].double().cpu().numpy()
            x = x * np.repeat(sc, B, axis=1)
        rows = np.zeros((T * k, K))
        rows[:source.size] = x[source]
        out = {"rows": rows}
        if c["dtype"] == "e4m3":
            out["scales"] = np.zeros((T * k, K // B))
            out["scales"][:source.size] = sc[source]
        return out | {"offsets": None, "inv": None}
    slots = [(s["inv"][:, j] >= 0).nonzero().squeeze(1) for j in range(k)]  # tokens whose j-th slot stays
    row = lambda j: s["inv"][slots[j], j].long()  # noqa: E731
    weight = lambda j: 1.0 if s["weights"] is None else s["weights"][slots[j], j].double().unsqueeze(1)  # noqa: E731
    if not c["back"]:
        out = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        for j in range(k):
            out[slots[j]] += s["y"][row(j)].double() * weight(j)
        return {"out": out.cpu().numpy()}
    dy, dw = torch.zeros(T * k, K, dtype=torch.float64, device="cuda"), torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        d = s["dout"][slots[j]].double()
        dy[row(j)] = d * weight(j)
        dw[slots[j], j] = torch.einsum("tk,tk->t", d, s["y"][row(j)].double())
    dy = dy.cpu().numpy()
    return {"dy": dy} if s["weights"] is None else {"dy": dy, "dweights": dw.cpu().numpy()}
