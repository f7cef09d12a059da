"""Measured cases of the mixture-of-experts and 8-bit integer operators.

Four operators of a quantized mixture-of-experts step:

  route    w4a16_moe_route     router scores -> chosen experts, weights and the rows of each expert
  experts  w4a16_gemm_experts  the experts' products with 4-bit weights over the rows routed to them
  combine  w4a16_moe_combine   the experts' outputs back into token order, weighted, plus a base
  int8     w8a8_gemm           8-bit integer product, a scale per row and per output channel

`run` computes them in plain torch operations, or, where `own` is set, with the framework's calls.
Weights are made directly in the packed arrangements of include/w4a16.h.
"""
import math

import torch

own = False

# Position of k offset i (0..15) inside a stored 16-block of int8 codes is
# ORDER.index(i): byte j of a block holds the code of offset ORDER[j].
ORDER = [0, 4, 1, 5, 2, 6, 3, 7, 8, 12, 9, 13, 10, 14, 11, 15]


def listed():
    """Hidden size 5120 and the 4-bit group of 128 are the decode layer set's; dense int8 shapes
    are its projections. 128 experts of width 1024 (256 for routing alone), 8 per token."""
    return [
        # one token of one stream: pure latency
        {"name": "route-1", "op": "route", "T": 1, "E": 128, "k": 8, "scoring": "softmax",
         "groups": 1, "kept": 1, "top": 1, "renorm": True, "scale": 1.0, "bias": False,
         "half": False, "pad": 0},
        # a decode batch padded to a captured graph's 64 rows, group-limited with a balance bias
        {"name": "route-64-groups", "op": "route", "T": 64, "E": 256, "k": 8, "scoring": "sigmoid",
         "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5, "bias": True,
         "half": True, "pad": 3},
        # a prefill batch of many prompts
        {"name": "route-8191-groups", "op": "route", "T": 8191, "E": 256, "k": 8,
         "scoring": "sigmoid", "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5,
         "bias": True, "half": False, "pad": 0},
        # single-stream decode: gate and up of the 8 chosen experts, SwiGLU in the epilogue
        {"name": "experts-gate-up-1", "op": "experts", "T": 1, "E": 128, "k": 8, "N": 2048,
         "K": 5120, "group": 128, "act": True, "shared_rows": True, "skew": 0.0},
        # the down product of a decode batch: every slot has its own row
        {"name": "experts-down-37", "op": "experts", "T": 37, "E": 128, "k": 8, "N": 5120,
         "K": 1024, "group": 128, "act": False, "shared_rows": False, "skew": 0.5},
        # batched serving: about 16 rows per expert, unevenly spread
        {"name": "experts-gate-up-256", "op": "experts", "T": 256, "E": 128, "k": 8, "N": 2048,
         "K": 5120, "group": 128, "act": True, "shared_rows": True, "skew": 0.5},
        # a prefill chunk: 256 rows per expert on average
        {"name": "experts-gate-up-4096", "op": "experts", "T": 4096, "E": 128, "k": 8, "N": 2048,
         "K": 5120, "group": 128, "act": True, "shared_rows": True, "skew": 0.5},
        # one token's weighted sum on top of the shared expert
        {"name": "combine-1", "op": "combine", "T": 1, "k": 8, "N": 5120, "base": True},
        # the same for a prefill chunk
        {"name": "combine-4096", "op": "combine", "T": 4096, "k": 8, "N": 5120, "base": True},
        # single-stream decode through the qkv projection
        {"name": "int8-qkv-1", "op": "int8", "M": 1, "N": 7168, "K": 5120},
        # batched decode through the down projection
        {"name": "int8-down-64", "op": "int8", "M": 64, "N": 5120, "K": 17408},
        # a prefill chunk through gate and up
        {"name": "int8-gate-up-1024", "op": "int8", "M": 1024, "N": 34816, "K": 5120},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "combine", "int8", "int8"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = rng.choice([8, 13, 16, 32]) if groups > 1 else _log(rng, 8, 256)
        E = groups * per
        kept = rng.randint(1, groups)
        T = _log(rng, 1, 8191)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, kept * per)),
                "scoring": rng.choice(["softmax", "sigmoid"]), "groups": groups, "kept": kept,
                "top": rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "scale": round(rng.uniform(0.5, 3.0), 2), "bias": rng.random() < 0.6,
                "half": rng.random() < 0.5, "pad": rng.choice([0, 0, T // 20])}
    if op == "experts":
        group = rng.choice([32, 64, 128, 128, 128])
        E = rng.choice([8, 16, 40, 64, 128])
        act = rng.random() < 0.5
        K = 128 * rng.randint(4, 40)
        N = 32 * rng.randint(16, 64) if act else _log(rng, 500, 5120)
        while E * N * K > 1.4e9:
            E //= 2
        T = _log(rng, 1, 4096)
        while 2 * N * K * T * 8 > 6.8e11:
            T = T // 2 + 1
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, E)), "N": N, "K": K,
                "group": group, "act": act, "shared_rows": act,
                "skew": rng.choice([0.0, 0.5, 1.0])}
    if op == "combine":
        return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, 8),
                "N": _log(rng, 257, 5120), "base": rng.random() < 0.5}
    M, N, K = _log(rng, 1, 1024), _log(rng, 500, 34816), 16 * _log(rng, 16, 1088)
    while 2 * M * N * K > 3.6e11:
        M, N = M // 2 + 1, N // 2 + 1
    return {"op": op, "M": M, "N": N, "K": K}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    op = case["op"]
    s = {"case": case}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        logits = torch.randn(T, E, generator=g, device=dev) * 1.5
        if case["pad"]:
            logits[T - case["pad"]:] = -math.inf  # padding tokens go nowhere
        s["logits"] = logits.to(torch.bfloat16) if case["half"] else logits
        s["bias"] = torch.randn(E, generator=g, device=dev) * 0.05 if case["bias"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        s["rows"] = torch.empty(T * k, dtype=torch.int32, device=dev)
        if own:
            import w4a16_weight_only_gemm_amd as w4
            n = w4.w4a16_moe_route_workspace_bytes(T, E)
            s["workspace"] = torch.empty(max(n, 4) // 4, dtype=torch.int32, device=dev)
    elif op == "experts":
        T, E, k, N, K, grp = (case[n] for n in ("T", "E", "k", "N", "K", "group"))
        blocks, G = (N + 15) // 16, K // grp
        R = T * k
        x_rows = T if case["shared_rows"] else R
        s["x"] = torch.randn(x_rows, K, generator=g, device=dev).to(torch.bfloat16)
        # every 32-bit pattern is eight codes
        s["qweight"] = torch.randint(-2**31, 2**31, (E, blocks, G, 64, grp // 32), generator=g,
                                     device=dev, dtype=torch.int32)
        sc = (torch.rand(E, blocks, G, 16, generator=g, device=dev) + 0.5) / (4 * math.sqrt(K))
        s["scales"] = sc.to(torch.float16)
        fav = torch.randn(E, generator=g, device=dev) * case["skew"]
        score = torch.randn(T, E, generator=g, device=dev) + fav
        ids = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k].reshape(-1)
        s["slot_expert"] = ids
        s["rows"] = torch.sort(ids, stable=True).indices.to(torch.int32)
        count = torch.bincount(ids, minlength=E)
        s["offsets"] = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)]).to(torch.int32)
        s["most"] = int(count.max())  # the plain form's batch height
        s["y"] = torch.empty(R, N // 2 if case["act"] else N, dtype=torch.bfloat16, device=dev)
    elif op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        s["y"] = torch.randn(T * k, N, generator=g, device=dev).to(torch.bfloat16)
        w = torch.rand(T, k, generator=g, device=dev) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["ids"] = torch.randint(0, 128, (T, k), generator=g, device=dev, dtype=torch.int32)
        s["base"] = (torch.randn(T, N, generator=g, device=dev).to(torch.bfloat16)
                     if case["base"] else None)
        s["out"] = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        blocks, steps = (N + 15) // 16, (K + 63) // 64
        x = torch.randn(M, K, generator=g, device=dev)
        big = x.abs().amax(1, keepdim=True)
        s["xq"] = torch.round(x * (127 / big)).to(torch.int8)
        s["sx"] = (big / 127).reshape(M).contiguous()
        # weights of a normal distribution quantized per channel; the arrangement is a permutation,
        # so independent codes can be drawn in place; k at or past K is zero
        w = torch.randn(blocks, steps, 64, 16, generator=g, device=dev)
        w = torch.round(w * 31).clamp_(-127, 127).to(torch.int8)
        if K % 64:
            w[:, steps - 1, 16 * (K % 64 // 16):] = 0
        s["qweight"] = w
        s["scales"] = (torch.rand(N, generator=g, device=dev) + 0.5) / (32 * math.sqrt(K))
        s["y"] = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    z = s["logits"].double()
    open_ = ~(torch.isnan(z) | (z == -math.inf))
    low = torch.full_like(z, -math.inf)
    if c["scoring"] == "softmax":
        m = torch.where(open_, z, low).amax(1, keepdim=True)
        e = torch.where(open_, torch.exp(z - m), torch.zeros_like(z))
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
        pick = z  # the same order as the scores, and exact
    else:
        score = torch.where(open_, 1 / (1 + torch.exp(-z)), torch.zeros_like(z))
        pick = z
    if s["bias"] is not None or c["groups"] > 1:
        pick = score if s["bias"] is None else score + s["bias"].double()
    pick = torch.where(open_, pick, low)
    if c["groups"] > 1:
        best = torch.sort(pick.view(T, c["groups"], -1), dim=2, descending=True).values
        best = best[:, :, :c["top"]]
        some = best[:, :, 0] > -math.inf
        value = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        value = torch.where(some, value, torch.full_like(value, -math.inf))
        order = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        keep = keep.repeat_interleave(E // c["groups"], dim=1)
        pick = torch.where(keep, pick, low)
    best = torch.sort(pick, dim=1, descending=True, stable=True)
    ids, there = best.indices[:, :k], best.values[:, :k] > -math.inf
    w = torch.where(there, score.gather(1, ids), torch.zeros_like(score[:, :k]))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    ids = torch.where(there, ids, torch.full_like(ids, -1))
    key = torch.where(ids < 0, torch.full_like(ids, E), ids).reshape(-1)
    order = torch.sort(key, stable=True)
    rows = torch.where(order.values < E, order.indices, torch.full_like(order.indices, -1))
    edges = torch.arange(E + 1, device=z.device)
    offsets = (key.view(1, -1) < edges.view(-1, 1)).sum(1)
    return (ids.to(torch.int32), (w * c["scale"]).float(), offsets.to(torch.int32),
            rows.to(torch.int32))


def _codes4(words):
    """int32 words [...] -> fp32 codes [..., 8] in k order (nibble i/2 + 4 (i%2) holds k = i)."""
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=words.device, dtype=torch.int32)
    c = (words.unsqueeze(-1) >> shift) & 15
    return ((c ^ 8) - 8).float()


def _weights4(qweight, scales):
    """Packed [e][blocks][G][64][wpl] and [e][blocks][G][16] -> fp32 [e][blocks * 16][K]."""
    e, blocks, G, _, wpl = qweight.shape
    w = _codes4(qweight.view(e, blocks, G, 4, 16, wpl)).view(e, blocks, G, 4, 16, wpl * 8)
    w = w * scales.float().view(e, blocks, G, 1, 16, 1)
    return w.permute(0, 1, 4, 2, 3, 5).reshape(e, blocks * 16, G * 4 * wpl * 8)


def _plain_experts(s):
    c = s["case"]
    E, k, N = c["E"], c["k"], c["N"]
    ids, R = s["slot_expert"], c["T"] * c["k"]
    x = s["x"].float()
    if c["shared_rows"]:
        x = x.repeat_interleave(k, dim=0)
    if R <= E:
        w = _weights4(s["qweight"][ids], s["scales"][ids])  # one matrix per slot
        y = torch.bmm(w, x.view(R, -1, 1)).view(R, -1)[:, :N]
    else:
        w = _weights4(s["qweight"], s["scales"])
        rows = s["rows"].long()
        e = ids[rows]
        at = e * s["most"] + torch.arange(R, device=x.device) - s["offsets"].long()[e]
        xp = x.new_zeros(E * s["most"], x.shape[1]).index_copy_(0, at, x[rows])
        yp = torch.bmm(xp.view(E, s["most"], -1), w.transpose(1, 2)).view(E * s["most"], -1)
        y = yp.new_empty(R, N).index_copy_(0, rows, yp[at][:, :N])
    if c["act"]:
        a, b = y[:, :N // 2], y[:, N // 2:]
        y = a / (1 + torch.exp(-a)) * b
    return y.to(torch.bfloat16)


def _plain_combine(s):
    c = s["case"]
    y = s["y"].float().view(c["T"], c["k"], c["N"])
    w = torch.where(s["ids"] < 0, torch.zeros_like(s["weights"]), s["weights"])
    out = (y * w.unsqueeze(2)).sum(1)
    if s["base"] is not None:
        out = out + s["base"].float()
    return out.to(torch.bfloat16)


def _codes8(packed, N, K):
    """Packed int8 [blocks][steps][64][16] -> [N][K] in k order."""
    blocks, steps = packed.shape[:2]
    w = packed.view(blocks, steps, 4, 16, 16).permute(0, 3, 1, 2, 4)
    w = w.reshape(blocks * 16, steps * 4, 16)
    back = torch.tensor([ORDER.index(i) for i in range(16)], device=packed.device)
    return w[:, :, back].reshape(blocks * 16, steps * 64)[:N, :K]


def _plain_int8(s):
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    w = _codes8(s["qweight"], N, K).double()  # sums pass what 32 bits hold exactly
    back = torch.tensor([ORDER.index(i) for i in range(16)], device=w.device)
    x = s["xq"].view(M, K // 16, 16)[:, :, back].reshape(M, K).double()
    y = torch.mm(x, w.t()) * s["sx"].double().view(M, 1) * s["scales"].double()
    return y.float().to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import w4a16_weight_only_gemm_amd as w4
        if op == "route":
            w4.w4a16_moe_route(
                s["logits"], s["bias"], c["T"], c["E"], c["k"], s["ids"], s["weights"],
                s["offsets"], s["rows"], s["workspace"],
                scoring=(w4.W4A16_ROUTE_SOFTMAX if c["scoring"] == "softmax"
                         else w4.W4A16_ROUTE_SIGMOID),
                groups=c["groups"], groups_kept=c["kept"], group_top=c["top"],
                renormalize=c["renorm"], scale=c["scale"])
            return s["ids"], s["weights"], s["offsets"], s["rows"]
        if op == "experts":
            w4.w4a16_gemm_experts(
                s["x"], s["qweight"], s["scales"], s["y"], s["rows"], s["offsets"],
                c["T"] * c["k"], c["E"], c["k"] if c["shared_rows"] else 1, c["N"], c["K"],
                c["group"], act=w4.W4A16_ACT_SWIGLU if c["act"] else w4.W4A16_ACT_NONE)
            return s["y"]
        if op == "combine":
            w4.w4a16_moe_combine(s["y"], s["ids"], s["weights"], s["base"], s["out"], c["T"],
                                 c["k"], c["N"])
            return s["out"]
        w4.w8a8_gemm(s["xq"], s["sx"], s["qweight"], s["scales"], s["y"], c["M"], c["N"], c["K"])
        return s["y"]
    if op == "route":
        return _plain_route(s)
    if op == "experts":
        return _plain_experts(s)
    if op == "combine":
        return _plain_combine(s)
    return _plain_int8(s)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * (2 if case["half"] else 4) + T * k * 12 + 4 * (E + 1) + (4 * E if case["bias"] else 0)
        return {"bytes": b, "flops": T * E * 4}
    if op == "experts":
        T, E, k, N, K, g = (case[n] for n in ("T", "E", "k", "N", "K", "group"))
        active = E * (1 - (1 - k / E) ** T)  # expected over even routing
        weights = active * ((N + 15) // 16 * 16) * (K / 2 + 2 * K / g)
        x_rows = T if case["shared_rows"] else T * k
        out = T * k * (N // 2 if case["act"] else N)
        return {"bytes": int(weights + 2 * x_rows * K + 2 * out + 4 * T * k + 4 * E),
                "flops": 2 * T * k * N * K}
    if op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        return {"bytes": 2 * T * N * (k + 1 + (1 if case["base"] else 0)) + 8 * T * k,
                "flops": 2 * T * k * N}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": N * K + M * K + 4 * (M + N) + 2 * M * N, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ 64-bit definitions

def _exact_route(s):
    import numpy as np
    c = s["case"]
    z = s["logits"].double().cpu().numpy()
    T, E, k = c["T"], c["E"], c["k"]
    live = np.isfinite(z) | (z == np.inf)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if c["scoring"] == "softmax":
            p = np.where(live, np.exp(z - np.max(np.where(live, z, -np.inf), axis=1, keepdims=True)), 0.0)
            p = p / np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
        else:
            p = np.where(live, 1.0 / (1.0 + np.exp(-z)), 0.0)
    v = p if s["bias"] is None else p + s["bias"].double().cpu().numpy()[None]
    if s["bias"] is None and c["groups"] == 1:
        v = z
    v = np.where(live, v, -np.inf)
    if c["groups"] > 1:
        part = -np.sort(-v.reshape(T, c["groups"], -1), axis=2)[:, :, :c["top"]]
        value = np.where(np.isinf(part), 0.0, part).sum(axis=2)
        value = np.where(np.isinf(part[:, :, 0]), -np.inf, value)
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        v = np.where(np.repeat(rank < c["kept"], E // c["groups"], axis=1), v, -np.inf)
    ids = np.argsort(-v, axis=1, kind="stable")[:, :k]
    got = np.take_along_axis(v, ids, 1) > -np.inf
    w = np.where(got, np.take_along_axis(p, ids, 1), 0.0)
    if c["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    ids = np.where(got, ids, -1)
    flat = ids.reshape(-1)
    slots = np.nonzero(flat >= 0)[0]
    rows = np.full(T * k, -1)
    rows[:slots.size] = slots[np.argsort(flat[slots], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[slots], minlength=E))])
    return (ids.astype(np.int32), w * c["scale"], offsets.astype(np.int32), rows.astype(np.int32))


def _exact_experts(s):
    c = s["case"]
    E, k, N, K, g = c["E"], c["k"], c["N"], c["K"], c["group"]
    wpl = g // 32
    dev = s["x"].device
    n = torch.arange(N, device=dev)
    kk = torch.arange(K, device=dev)
    # where the code of (n, k) sits: word j = k / 8 of column n, nibble i / 2 + 4 (i % 2)
    j, i = kk // 8, kk % 8
    tile, inside = j // (g // 8), j % (g // 8)
    lane_part, word = inside // wpl, inside % wpl
    nib = i // 2 + 4 * (i % 2)
    pos = ((n // 16).view(-1, 1) * (K // g) + tile.view(1, -1)) * 64
    pos = (pos + lane_part.view(1, -1) * 16 + (n % 16).view(-1, 1)) * wpl + word.view(1, -1)
    spos = ((n // 16).view(-1, 1) * (K // g) + (kk // g).view(1, -1)) * 16 + (n % 16).view(-1, 1)
    out = torch.empty(c["T"] * k, N, dtype=torch.float64, device=dev)
    slots, edge = s["rows"].long(), s["offsets"].tolist()
    for e in range(E):
        mine = slots[edge[e]:edge[e + 1]]
        if mine.numel() == 0:
            continue
        code = (s["qweight"][e].reshape(-1)[pos].long() >> (4 * nib).view(1, -1)) & 15
        code = torch.where(code > 7, code - 16, code).double()
        w = code * s["scales"][e].reshape(-1)[spos].double()
        src = mine // k if c["shared_rows"] else mine
        out[mine] = s["x"][src].double() @ w.t()
    if c["act"]:
        a, b = out[:, :N // 2], out[:, N // 2:]
        out = a * torch.sigmoid(a) * b
    return out


def _exact_combine(s):
    c = s["case"]
    w = (s["weights"] * (s["ids"] >= 0)).double()
    out = torch.bmm(w.view(c["T"], 1, c["k"]), s["y"].double().view(c["T"], c["k"], c["N"]))
    out = out.view(c["T"], c["N"])
    return out if s["base"] is None else out + s["base"].double()


def _exact_int8(s):
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    dev = s["xq"].device
    kk = torch.arange(K, device=dev)
    byte = torch.tensor([ORDER.index(i) for i in range(16)], device=dev)[kk % 16]
    n = torch.arange(N, device=dev).view(-1, 1)
    steps = (K + 63) // 64
    pos = ((n // 16 * steps + (kk // 64)) * 64 + kk % 64 // 16 * 16 + n % 16) * 16 + byte
    w = s["qweight"].reshape(-1)[pos].double()
    x = s["xq"][:, kk // 16 * 16 + byte].double()
    return (x @ w.t()) * torch.outer(s["sx"].double(), s["scales"].double())


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "combine": _exact_combine,
            "int8": _exact_int8}[case["op"]](s)
