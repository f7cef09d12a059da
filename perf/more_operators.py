"""Measured cases of the operators that join a decoder layer's 4-bit products.

Three operators of a layer whose weights are held in 4 bits:

  epilogue   w4a16_gemm_epilogue  the 4-bit product with bias, activation (gated ones too), scale
                                  and residual in its epilogue
  norm       w4a16_norm           a block's output normalised, gated, scaled and added to the
                                  residual stream, and the next block's norm of the sum, as bf16
                                  or as the 8-bit codes of w4a8_quantize
  moe_layer  w4a16_moe_layer      a whole mixture-of-experts layer for a few tokens: the router's
                                  product, the choice, the experts and the weighted sum

`run` computes them in plain torch operations, or, where `own` is set, with the framework's calls.
Weights are made directly in the packed arrangement of include/w4a16.h.
"""
import math

import torch

own = False

# Position of k offset i (0..15) inside a stored 16-block of int8 codes is
# ORDER.index(i): byte j of a block holds the code of offset ORDER[j].
ORDER = [0, 4, 1, 5, 2, 6, 3, 7, 8, 12, 9, 13, 10, 14, 11, 15]


def listed():
    """Products are the decode layer set's (hidden size 5120, group 128); experts are 128 of width
    1024 with 8 per token, 256 of half that width in groups, and 32 small ones."""
    return [
        # single-stream decode: the qkv projection of a model with biases
        {"name": "epilogue-qkv-1-bias", "op": "epilogue", "M": 1, "N": 7168, "K": 5120,
         "group": 128, "act": "none", "bias": True, "residual": False, "scale": 1.0},
        # a speculative block of 16 positions through gate and up
        {"name": "epilogue-gate-up-16-swiglu", "op": "epilogue", "M": 16, "N": 34816, "K": 5120,
         "group": 128, "act": "swiglu", "bias": False, "residual": False, "scale": 1.0},
        # a decode batch through the down projection, onto the residual stream
        {"name": "epilogue-down-64-residual", "op": "epilogue", "M": 64, "N": 5120, "K": 17408,
         "group": 128, "act": "none", "bias": False, "residual": True, "scale": 0.5},
        # batched serving, gate and up of 1024 rows
        {"name": "epilogue-gate-up-1024-swiglu", "op": "epilogue", "M": 1024, "N": 34816,
         "K": 5120, "group": 128, "act": "swiglu", "bias": False, "residual": False,
         "scale": 1.0},
        # one token between two blocks: add to the residual stream, norm for the next block
        {"name": "norm-1", "op": "norm", "T": 1, "N": 5120, "kind": "rms", "post": False,
         "gate": 0, "scale": 1.0, "unit": False, "wide": False, "codes": False},
        # a decode batch whose next products take 8-bit activations
        {"name": "norm-64-post-codes", "op": "norm", "T": 64, "N": 5120, "kind": "rms",
         "post": True, "gate": 0, "scale": 1.0, "unit": True, "wide": False, "codes": True},
        # a prefill chunk of an odd number of rows with norms on both sides of the block
        {"name": "norm-4095-post", "op": "norm", "T": 4095, "N": 5120, "kind": "rms", "post": True,
         "gate": 0, "scale": 0.7, "unit": False, "wide": True, "codes": False},
        # layer norms of conditioned blocks: a gate per sequence of 256 rows, rows of odd length
        {"name": "norm-2048-gated-odd", "op": "norm", "T": 2048, "N": 2741, "kind": "layer",
         "post": True, "gate": 256, "scale": 1.0, "unit": False, "wide": False, "codes": False},
        # single-stream decode through a whole layer of experts
        {"name": "moe-layer-1", "op": "moe_layer", "T": 1, "E": 128, "k": 8, "H": 5120, "I": 1024,
         "group": 128, "scoring": "softmax", "groups": 1, "kept": 1, "top": 1, "renorm": True,
         "scale": 1.0, "bias": False, "half": True, "base": True, "pad": 0},
        # a speculative block, experts chosen within groups
        {"name": "moe-layer-4-groups", "op": "moe_layer", "T": 4, "E": 256, "k": 8, "H": 5120,
         "I": 512, "group": 128, "scoring": "sigmoid", "groups": 8, "kept": 4, "top": 2,
         "renorm": True, "scale": 2.5, "bias": True, "half": False, "base": True, "pad": 0},
        # a small model's layer, finer groups of weights
        {"name": "moe-layer-3-small", "op": "moe_layer", "T": 3, "E": 32, "k": 4, "H": 2048,
         "I": 768, "group": 64, "scoring": "softmax", "groups": 1, "kept": 1, "top": 1,
         "renorm": False, "scale": 1.0, "bias": False, "half": False, "base": True, "pad": 0},
        # a decode batch in a graph captured for 16 rows, three of them padding
        {"name": "moe-layer-16-padded", "op": "moe_layer", "T": 16, "E": 128, "k": 8, "H": 5120,
         "I": 1024, "group": 128, "scoring": "softmax", "groups": 1, "kept": 1, "top": 1,
         "renorm": True, "scale": 1.0, "bias": False, "half": True, "base": True, "pad": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["epilogue", "norm", "moe_layer"])
    if op == "epilogue":
        group = rng.choice([32, 64, 128, 128, 128, 256])
        K = group * max(1, _log(rng, 512, 17408) // group)
        act = rng.choice(["none", "none", "swiglu", "geglu", "silu", "gelu", "gelu_tanh", "relu"])
        N = _log(rng, 300, 34816)
        if act in ("swiglu", "geglu"):
            N = 32 * max(1, N // 32)
        while N * K > 1.78e8:
            N = 32 * (N // 64)
        M = _log(rng, 1, 1024)
        return {"op": op, "M": M, "N": N, "K": K, "group": group, "act": act,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5,
                "scale": rng.choice([1.0, 1.0, 0.5, round(rng.uniform(0.1, 2.0), 2)])}
    if op == "norm":
        codes = rng.random() < 0.3
        N = _log(rng, 128, 17408)
        N = N // 16 * 16 if codes else N
        T = _log(rng, 1, 8192)
        while T * N > 4095 * 5120:
            T = T // 2 + 1
        return {"op": op, "T": T, "N": N, "kind": rng.choice(["rms", "rms", "layer"]),
                "post": rng.random() < 0.5, "gate": rng.choice([0, 0, 1, 37, T]),
                "scale": rng.choice([1.0, round(rng.uniform(0.1, 2.0), 2)]),
                "unit": rng.random() < 0.3, "wide": rng.random() < 0.3, "codes": codes}
    group = rng.choice([32, 64, 128, 128, 128, 256])
    groups = rng.choice([1, 1, 4, 8])
    E = groups * rng.choice([8, 16, 32]) if groups > 1 else rng.choice([8, 16, 40, 64, 128])
    kept = rng.randint(1, groups)
    H, I = 256 * rng.randint(4, 20), 256 * rng.randint(1, 6)
    while E * H * I > 128 * 5120 * 1024:
        I = 256 * max(1, I // 512) if I > 256 else I
        H = 256 * (H // 512) if I == 256 else H
    T = _log(rng, 1, 16)
    return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, kept * (E // groups))), "H": H,
            "I": I, "group": group, "scoring": rng.choice(["softmax", "sigmoid"]),
            "groups": groups, "kept": kept, "top": rng.choice([1, 2]),
            "renorm": rng.random() < 0.7, "scale": round(rng.uniform(0.5, 2.5), 2),
            "bias": rng.random() < 0.5, "half": rng.random() < 0.5, "base": True,
            "pad": rng.choice([0, 0, T // 4])}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _packed(g, lead, N, K, group, size=1.0):
    """Packed random weights [*lead][blocks][G][64][wpl] and scales [*lead][blocks][G][16]."""
    blocks, G = (N + 15) // 16, K // group
    # every 32-bit pattern is eight codes
    q = torch.randint(-2**31, 2**31, (*lead, blocks, G, 64, group // 32), generator=g,
                      device="cuda", dtype=torch.int32)
    s = (torch.rand(*lead, blocks, G, 16, generator=g, device="cuda") + 0.5) * size
    return q, (s / (4 * math.sqrt(K))).to(torch.float16)


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    bf16 = torch.bfloat16

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        n_out = N // 2 if case["act"] in ("swiglu", "geglu") else N
        s["x"] = randn(M, K).to(bf16)
        s["qweight"], s["scales"] = _packed(g, (), N, K, case["group"])
        s["bias"] = (randn(N) * 0.5).to(bf16) if case["bias"] else None
        s["residual"] = randn(M, n_out).to(bf16) if case["residual"] else None
        s["y"] = torch.empty(M, n_out, dtype=bf16, device=dev)
    elif case["op"] == "norm":
        T, N = case["T"], case["N"]
        layer, codes = case["kind"] == "layer", case["codes"]
        wide = torch.float32 if case["wide"] else bf16
        centre = 0.0 if case["unit"] else 1.0  # weights are held as their difference from one
        s["y"] = (randn(T, N) * torch.exp(randn(T, 1))).to(bf16)
        s["residual"] = (randn(T, N) * 3 + (randn(T, 1) if layer else 0)).to(wide)
        s["weight"] = (randn(N) * 0.2 + centre).to(bf16)
        s["bias"] = (randn(N) * 0.2).to(bf16) if layer else None
        s["post_weight"] = (randn(N) * 0.2 + centre).to(bf16) if case["post"] else None
        s["post_bias"] = (randn(N) * 0.2).to(bf16) if case["post"] and layer else None
        rows = case["gate"]
        s["gate"] = (randn((T + rows - 1) // rows, N) * 0.5).to(bf16) if rows else None
        s["residual_out"] = torch.empty(T, N, dtype=wide, device=dev)
        s["x"] = torch.empty(T, N, dtype=bf16, device=dev)
        s["xq"] = torch.empty(T, N, dtype=torch.int8, device=dev) if codes else None
        s["sx"] = torch.empty(T, 1, dtype=torch.float32, device=dev) if codes else None
    else:
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["x"] = randn(T, H).to(bf16)
        router = randn(E, H) * (1.5 / math.sqrt(H))
        s["router"] = router.to(bf16) if case["half"] else router
        s["route_bias"] = randn(E) * 0.05 if case["bias"] else None
        s["gate_up"], s["gate_up_scales"] = _packed(g, (E,), 2 * I, H, case["group"])
        s["down"], s["down_scales"] = _packed(g, (E,), H, I, case["group"], 3.0)
        s["base"] = randn(T, H).to(bf16) if case["base"] else None
        live = torch.ones(T, dtype=torch.int32, device=dev)
        live[T - case["pad"]:] = 0
        s["live"] = live if case["pad"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        s["out"] = torch.empty(T, H, dtype=bf16, device=dev)
        if own:
            import w4a16_weight_only_gemm_amd as w4
            n = w4.w4a16_moe_layer_workspace_bytes(T, E, k, H, I)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

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


def _silu(v):
    return v / (1 + torch.exp(-v))


def _gelu_tanh(v):
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _plain_epilogue(s):
    c = s["case"]
    N, act = c["N"], c["act"]
    w = _weights4(s["qweight"].unsqueeze(0), s["scales"].unsqueeze(0))[0]
    p = torch.mm(s["x"].float(), w.t())[:, :N]
    if s["bias"] is not None:
        p = p + s["bias"].float()
    if act == "swiglu":
        p = _silu(p[:, :N // 2]) * p[:, N // 2:]
    elif act == "geglu":
        p = _gelu_tanh(p[:, :N // 2]) * p[:, N // 2:]
    elif act == "silu":
        p = _silu(p)
    elif act == "gelu":
        p = 0.5 * p * (1 + torch.erf(p / math.sqrt(2)))
    elif act == "gelu_tanh":
        p = _gelu_tanh(p)
    elif act == "relu":
        p = p.clamp_min(0)
    p = p * c["scale"]
    if s["residual"] is not None:
        p = p + s["residual"].float()
    return p.to(torch.bfloat16)


EPS = 1e-6


def _normed(v, c, weight, bias):
    if c["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    v = v * (weight.float() + 1 if c["unit"] else weight.float())
    return v if bias is None else v + bias.float()


def _plain_norm(s):
    c = s["case"]
    u = s["y"].float()
    if c["post"]:
        u = _normed(u, c, s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        u = u * s["gate"].float().repeat_interleave(c["gate"], dim=0)[:c["T"]]
    r = s["residual"].float() + c["scale"] * u
    x = _normed(r, c, s["weight"], s["bias"])
    out = [r.to(s["residual"].dtype)]
    if not c["codes"]:
        return out + [x.to(torch.bfloat16)]
    big = x.abs().amax(1, keepdim=True)
    q = torch.round(x * (127 / big)).clamp(-127, 127)
    order = torch.tensor(ORDER, device=x.device)
    q = q.view(c["T"], -1, 16)[:, :, order].reshape(c["T"], -1)
    return out + [(q * (big / 127)).to(torch.bfloat16)]


def _choose(z, s):
    """Experts and weights from 64-bit logits (-inf in the rows of padding tokens)."""
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    low = torch.full_like(z, -math.inf)
    open_ = z > -math.inf
    if c["scoring"] == "softmax":
        e = torch.where(open_, torch.exp(z - z.amax(1, keepdim=True)), torch.zeros_like(z))
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1 / (1 + torch.exp(-z))
    pick = z
    if s["route_bias"] is not None or c["groups"] > 1:
        pick = score if s["route_bias"] is None else score + s["route_bias"].double()
        pick = torch.where(open_, pick, low)
    if c["groups"] > 1:
        best = torch.sort(pick.view(T, c["groups"], -1), dim=2, descending=True).values
        value = best[:, :, :c["top"]].sum(2)
        order = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        pick = torch.where(keep.repeat_interleave(E // c["groups"], dim=1), pick, low)
    best = torch.sort(pick, dim=1, descending=True, stable=True)
    ids, there = best.indices[:, :k], best.values[:, :k] > -math.inf
    w = torch.where(there, score.gather(1, ids), torch.zeros_like(score[:, :k]))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return torch.where(there, ids, torch.full_like(ids, -1)), w * c["scale"]


def _plain_moe_layer(s):
    c = s["case"]
    T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
    x = s["x"].double()
    z = torch.mm(x, s["router"].double().t())
    if s["live"] is not None:
        z = torch.where(s["live"].view(T, 1) != 0, z, torch.full_like(z, -math.inf))
    ids, w = _choose(z, s)
    at = ids.clamp_min(0).reshape(-1)
    # the weights of one matrix per slot for few slots, else of every expert
    few = T * k <= E // 2
    pick = at if few else torch.arange(E, device=at.device)
    gu = _weights4(s["gate_up"][pick], s["gate_up_scales"][pick])
    xf = s["x"].float()
    if few:
        p = torch.bmm(gu, xf.repeat_interleave(k, dim=0).view(T * k, H, 1)).view(T * k, 2 * I)
    else:
        p = torch.matmul(gu, xf.t().contiguous())[at, :, torch.arange(T * k, device=at.device) // k]
    h = _silu(p[:, :I]) * p[:, I:]
    dn = _weights4(s["down"][pick], s["down_scales"][pick])
    if few:
        y = torch.bmm(dn, h.view(T * k, I, 1)).view(T, k, H)
    else:
        # each expert's columns: the tokens that chose it, elsewhere zeros
        hp = h.new_zeros(E, I, T)
        token = torch.arange(T * k, device=at.device) // k
        hp[at, :, token] = torch.where(ids.reshape(-1, 1) >= 0, h, torch.zeros_like(h))
        y = torch.bmm(dn, hp)[at, :, token].view(T, k, H)
    out = (y * torch.where(ids >= 0, w, torch.zeros_like(w)).float().unsqueeze(2)).sum(1)
    if s["base"] is not None:
        out = out + s["base"].float()
    return out.to(torch.bfloat16), ids.to(torch.int32), w.float()


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if own:
        import w4a16_weight_only_gemm_amd as w4
        if c["op"] == "epilogue":
            w4.w4a16_gemm_epilogue(
                s["x"], s["qweight"], s["scales"], s["y"], c["M"], c["N"], c["K"], c["group"],
                bias=s["bias"], residual=s["residual"], scale=c["scale"],
                act=getattr(w4, "W4A16_ACT_" + c["act"].upper()))
            return s["y"]
        if c["op"] == "norm":
            w4.w4a16_norm(
                c["T"], c["N"], y=s["y"], residual=s["residual"], residual_out=s["residual_out"],
                post_norm=c["post"], post_weight=s["post_weight"], post_bias=s["post_bias"],
                gate=s["gate"], gate_rows=max(c["gate"], 1), scale=c["scale"], weight=s["weight"],
                bias=s["bias"], x=None if c["codes"] else s["x"], xq=s["xq"], sx=s["sx"],
                kind=w4.W4A16_NORM_LAYER if c["kind"] == "layer" else w4.W4A16_NORM_RMS, eps=EPS,
                unit_offset=c["unit"])
            if c["codes"]:  # what the codes stand for, in their stored order
                return s["residual_out"], torch.mul(s["xq"], s["sx"], out=s["x"])
            return s["residual_out"], s["x"]
        w4.w4a16_moe_layer(
            s["x"], s["router"], s["gate_up"], s["gate_up_scales"], s["down"], s["down_scales"],
            s["out"], s["ids"], s["weights"], c["T"], c["E"], c["k"], c["H"], c["I"], c["group"],
            s["workspace"], route_bias=s["route_bias"], base=s["base"], live=s["live"],
            scoring=(w4.W4A16_ROUTE_SOFTMAX if c["scoring"] == "softmax"
                     else w4.W4A16_ROUTE_SIGMOID),
            groups=c["groups"], groups_kept=c["kept"], group_top=c["top"],
            renormalize=c["renorm"], scale=c["scale"])
        return s["out"], s["ids"], s["weights"]
    if c["op"] == "epilogue":
        return _plain_epilogue(s)
    if c["op"] == "norm":
        return _plain_norm(s)
    return _plain_moe_layer(s)


def _weight_bytes(N, K, group):
    return ((N + 15) // 16 * 16) * (K // 2 + 2 * (K // group))


def work(case):
    if case["op"] == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        n_out = N // 2 if case["act"] in ("swiglu", "geglu") else N
        b = _weight_bytes(N, K, case["group"]) + 2 * M * K + 2 * M * n_out
        b += (2 * N if case["bias"] else 0) + (2 * M * n_out if case["residual"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    if case["op"] == "norm":
        T, N, rows = case["T"], case["N"], case["gate"]
        b = T * N * (2 + 2 * (4 if case["wide"] else 2) + (1 if case["codes"] else 2))
        vectors = (2 if case["kind"] == "layer" else 1) * (2 if case["post"] else 1)
        b += 2 * N * (vectors + ((T + rows - 1) // rows if rows else 0))
        return {"bytes": b + (4 * T if case["codes"] else 0), "flops": 12 * T * N}
    T, E, k, H, I, g = (case[n] for n in ("T", "E", "k", "H", "I", "group"))
    tokens = T - case["pad"]
    active = E * (1 - (1 - k / E) ** tokens)  # expected over even routing
    weights = active * (_weight_bytes(2 * I, H, g) + _weight_bytes(H, I, g))
    b = weights + E * H * (2 if case["half"] else 4) + 2 * T * H * (3 if case["base"] else 2)
    return {"bytes": int(b + 8 * T * k),
            "flops": 2 * T * E * H + 2 * tokens * k * 3 * H * I}


# ------------------------------------------------------------------ 64-bit definitions

def _exact_weights(qweight, scales, N, K, group):
    """fp64 [N][K] of one packed matrix: each code looked up at its place."""
    wpl = group // 32
    dev = qweight.device
    n = torch.arange(N, device=dev, dtype=torch.int32)
    kk = torch.arange(K, device=dev, dtype=torch.int32)
    # the code of (n, k): word j = k / 8 of column n, nibble i / 2 + 4 (i % 2)
    j, i = kk // 8, kk % 8
    tile, inside = j // (group // 8), j % (group // 8)
    lane_part, word = inside // wpl, inside % wpl
    nib = i // 2 + 4 * (i % 2)
    block = (n // 16).view(-1, 1) * (K // group)
    pos = ((block + tile.view(1, -1)) * 64 + lane_part.view(1, -1) * 16
           + (n % 16).view(-1, 1)) * wpl + word.view(1, -1)
    code = (qweight.reshape(-1)[pos] >> (4 * nib).view(1, -1)) & 15
    code = torch.where(code > 7, code - 16, code).double()
    del pos
    spos = (block + (kk // group).view(1, -1)) * 16 + (n % 16).view(-1, 1)
    return code.mul_(scales.reshape(-1)[spos].double())


def _exact_epilogue(s):
    c = s["case"]
    N, act = c["N"], c["act"]
    out = s["x"].double() @ _exact_weights(s["qweight"], s["scales"], N, c["K"], c["group"]).t()
    if s["bias"] is not None:
        out += s["bias"].double()
    gate = out[:, :N // 2] if act in ("swiglu", "geglu") else out
    if act in ("swiglu", "silu"):
        value = gate * torch.sigmoid(gate)
    elif act in ("geglu", "gelu_tanh"):
        value = gate * torch.sigmoid(1.5957691216057308 * (gate + 0.044715 * gate ** 3))
    elif act == "gelu":
        value = gate * torch.special.ndtr(gate)
    elif act == "relu":
        value = torch.maximum(gate, torch.zeros_like(gate))
    else:
        value = gate
    if act in ("swiglu", "geglu"):
        value = value * out[:, N // 2:]
    value = value * c["scale"]
    return value if s["residual"] is None else value + s["residual"].double()


def _exact_norm(s):
    import numpy as np
    c = s["case"]

    def host(t):
        return None if t is None else t.double().cpu().numpy()

    def norm(v, weight, bias):
        if c["kind"] == "layer":
            v = v - np.mean(v, axis=1)[:, None]
        v = v / np.sqrt(np.sum(v ** 2, axis=1)[:, None] / c["N"] + EPS)
        v = v * (host(weight) + (1.0 if c["unit"] else 0.0))[None]
        return v if bias is None else v + host(bias)[None]

    u = host(s["y"])
    if c["post"]:
        u = norm(u, s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        u = u * host(s["gate"])[np.arange(c["T"]) // c["gate"]]
    r = host(s["residual"]) + c["scale"] * u
    x = norm(r, s["weight"], s["bias"])
    if c["codes"]:
        unit = np.max(np.abs(x), axis=1, keepdims=True) / 127.0
        x = np.rint(x / unit) * unit
        x = x[:, np.arange(c["N"]) // 16 * 16 + np.array(ORDER)[np.arange(c["N"]) % 16]]
    return [r, x]


def _exact_moe_layer(s):
    import numpy as np
    c = s["case"]
    T, E, k, H, I, g = (c[n] for n in ("T", "E", "k", "H", "I", "group"))
    z = s["x"].double().cpu().numpy() @ s["router"].double().cpu().numpy().T
    out = torch.zeros(T, H, dtype=torch.float64, device=s["x"].device)
    if s["base"] is not None:
        out += s["base"].double()
    ids, weights = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T - c["pad"]):
        if c["scoring"] == "softmax":
            p = np.exp(z[t] - z[t].max())
            p = p / p.sum()
        else:
            p = 1.0 / (1.0 + np.exp(-z[t]))
        v = z[t]
        if s["route_bias"] is not None or c["groups"] > 1:
            v = p if s["route_bias"] is None else p + s["route_bias"].double().cpu().numpy()
        if c["groups"] > 1:
            part = -np.sort(-v.reshape(c["groups"], -1), axis=1)[:, :c["top"]]
            first = np.argsort(-part.sum(axis=1), kind="stable")[:c["kept"]]
            v = np.where(np.isin(np.arange(E) // (E // c["groups"]), first), v, -np.inf)
        ids[t] = np.argsort(-v, kind="stable")[:k]
        w = p[ids[t]]
        weights[t] = (w / w.sum() if c["renorm"] else w) * c["scale"]
    for e in np.unique(ids[ids >= 0]):
        gu = _exact_weights(s["gate_up"][e], s["gate_up_scales"][e], 2 * I, H, g)
        dn = _exact_weights(s["down"][e], s["down_scales"][e], H, I, g)
        for t, j in np.argwhere(ids == e):
            p = gu @ s["x"][t].double()
            out[t] += weights[t, j] * (dn @ (p[:I] * torch.sigmoid(p[:I]) * p[I:]))
    return out, ids.astype(np.int32), weights


def exact(case, seed):
    s = prepare(case, seed)
    return {"epilogue": _exact_epilogue, "norm": _exact_norm,
            "moe_layer": _exact_moe_layer}[case["op"]](s)
