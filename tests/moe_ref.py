"""Plain 64-bit definitions of the mixture-of-experts and W8A8 operators, on
NumPy arrays, written from include/w4a16_moe.h (no code shared with the
library), and the bounds the GPU tests hold results to."""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8   # one rounding to bf16, relative
F32 = 2.0 ** -24   # one rounding to fp32, relative
ORDER = [0, 4, 1, 5, 2, 6, 3, 7, 8, 12, 9, 13, 10, 14, 11, 15]


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bit patterns, nearest even (finite, infinite and NaN values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r).astype(np.uint16)


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def route(logits, bias, top_k, scoring="softmax", groups=1, groups_kept=1, group_top=1,
          renormalize=True, scale=1.0):
    """One token after the other, one choice after the other. Returns ids, weights
    (fp64), offsets, rows."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    big = float(np.finfo(np.float32).max)
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    per = E // groups
    for t in range(T):
        z = np.minimum(logits[t], big)
        live = np.array([not np.isnan(v) and v != -np.inf for v in z])
        score = np.zeros(E)
        if live.any():
            if scoring == "softmax":
                ex = np.exp(z[live] - z[live].max())
                score[live] = ex / ex.sum()
            else:
                with np.errstate(over="ignore"):
                    score[live] = 1.0 / (1.0 + np.exp(-z[live]))
        # scores grow with the logit; without bias and groups the logit decides exactly
        v = z if bias is None and groups == 1 else score + (0.0 if bias is None else np.asarray(bias, np.float64))
        allowed = live.copy()
        if groups > 1:
            value = []
            for g in range(groups):
                mine = sorted((v[e] for e in range(g * per, (g + 1) * per) if live[e]), reverse=True)
                value.append(sum(mine[:group_top]) if mine else -np.inf)
            best = sorted(range(groups), key=lambda g: (-value[g], g))[:groups_kept]
            for g in range(groups):
                if g not in best:
                    allowed[g * per:(g + 1) * per] = False
        order = sorted((e for e in range(E) if allowed[e]), key=lambda e: (-v[e], e))[:top_k]
        for j, e in enumerate(order):
            ids[t, j] = e
            weights[t, j] = score[e]
        if renormalize:
            total = weights[t].sum()
            weights[t] = weights[t] / total if total > 0 else 0.0
    weights = weights * scale
    lists = [[] for _ in range(E)]
    for s, e in enumerate(ids.reshape(-1)):
        if e >= 0:
            lists[e].append(s)
    offsets = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    rows = np.full(T * top_k, -1, np.int32)
    flat = [s for x in lists for s in x]
    rows[:len(flat)] = flat
    return ids, weights, offsets, rows


def experts(x, q, s, rows, offsets, x_div, group, swiglu=False):
    """x fp64 [.][K], q int8 [E][N][K], s fp64 [E][N][K / group]. Returns (y fp64
    [slots][out] with NaN where no list names the slot, bound of |result - y|).

    The bound counts the fp32 roundings of the kernels: within a group the
    biased products (24 + q) x are accumulated onto -24 sum(x), group + 2
    additions whose partial sums stay below S = sum (|24 + q| + 24) |x| of the
    group; the scaling rounds once more and G groups and up to 16 waves are
    added: (group + G + 20) half steps of S s in all. Then one rounding to
    bf16. SwiGLU: silu has slope at most 1.1 and magnitude at most |g|; the
    exponential, quotient and product add well under 64 half steps of fp32."""
    E, N, K = q.shape
    G = K // group
    out = N // 2 if swiglu else N
    slots = rows.size
    y = np.full((slots, out), np.nan)
    tol = np.zeros((slots, out))
    for e in range(E):
        mine = rows[offsets[e]:offsets[e + 1]]
        if mine.size == 0:
            continue
        xe = x[mine // x_div]
        se = np.repeat(s[e], group, axis=1)
        p = xe @ (q[e] * se).T
        mag = np.abs(xe) @ ((np.abs(24.0 + q[e]) + 24.0) * np.abs(se)).T
        d = (group + G + 20) * F32 * mag
        if swiglu:
            g, u = p[:, :out], p[:, out:]
            dg, du = d[:, :out], d[:, out:]
            with np.errstate(over="ignore"):
                sg = g / (1.0 + np.exp(-g))
            p = sg * u
            d = 1.1 * dg * (np.abs(u) + du) + np.abs(sg) * du + 64 * F32 * np.abs(p)
        y[mine] = p
        tol[mine] = d + BF16 * (np.abs(p) + d)
    return y, tol


def combine(y, ids, weights, base):
    """y fp64 [T * k][N]. Returns (out, bound): k + 1 fp32 additions and products
    below the sum of magnitudes, one rounding to bf16."""
    T, k = ids.shape
    N = y.shape[1]
    out = np.zeros((T, N)) if base is None else base.copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                term = weights[t, j] * y[t * k + j]
                out[t] += term
                mag[t] += np.abs(term)
    d = (k + 1) * F32 * mag
    return out, d + BF16 * (np.abs(out) + d)


def w8a8(xq, sx, q, sw):
    """Natural-order codes. The integer sum is exact; its conversion, the product
    of the scales and the product with it round to fp32, then to bf16."""
    acc = xq.astype(np.float64) @ q.astype(np.float64).T  # exact below 2^53
    y = acc * sx[:, None].astype(np.float64) * sw[None].astype(np.float64)
    return y, np.abs(y) * (BF16 * (1 + 4 * F32) + 4 * F32)


def arrange_codes(c: np.ndarray) -> np.ndarray:
    """Natural-order int8 [M][K] -> the stored order of w4a8_quantize."""
    M, K = c.shape
    return np.ascontiguousarray(c.reshape(M, K // 16, 16)[:, :, ORDER].reshape(M, K))


def w8a8_pack(q: np.ndarray) -> np.ndarray:
    """The packed arrangement, entry by entry."""
    N, K = q.shape
    blocks, steps = (N + 15) // 16, (K + 63) // 64
    out = np.zeros((blocks, steps, 64, 16), np.int8)
    for b in range(blocks):
        for t in range(steps):
            for lane in range(64):
                n, k = 16 * b + lane % 16, 64 * t + 16 * (lane // 16)
                if n < N and k < K:
                    out[b, t, lane] = q[n, k:k + 16][ORDER]
    return out.reshape(-1)


def check(got_bits: np.ndarray, ref: np.ndarray, tol: np.ndarray, what=""):
    """Every element within its bound, and the error's norm within one bf16 half
    step of the result's (single roundings reach about 0.4 of it)."""
    got = bf16_value(got_bits)
    assert np.isfinite(got).all(), what
    d = np.abs(got - ref)
    worst = np.max(d - tol) if d.size else 0.0
    assert worst <= 0, (what, float(worst), np.unravel_index(np.argmax(d - tol), d.shape))
    norm = np.linalg.norm(ref)
    if norm > 0:
        assert np.linalg.norm(got - ref) <= BF16 * norm, what
