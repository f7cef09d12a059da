"""Plain 64-bit definitions of the operators of include/w4a16_layer.h, on NumPy
arrays (no code shared with the library), and the bounds the GPU tests hold
results to: every rounding of the kernels counted as half a step, relative to
the value rounded, and carried through the steps that follow."""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

import moe_ref
from moe_ref import BF16, F32


def product(x, q, s, group):
    """x fp64 [M][K], q int8 [N][K], s fp64 [N][K / group]: (x W^T, bound), the bound
    that of moe_ref.experts: (group + G + 20) half steps of the biased sums."""
    K = q.shape[1]
    se = np.repeat(s, group, axis=1)
    mag = np.abs(x) @ ((np.abs(24.0 + q) + 24.0) * np.abs(se)).T
    return x @ (q * se).T, (group + K // group + 20) * F32 * mag


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def activation(v, act):
    if act in ("silu", "swiglu"):
        return v * _sigmoid(v)
    if act in ("gelu_tanh", "geglu"):
        return v * _sigmoid(2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3))
    if act == "gelu":
        return 0.5 * v * erfc(-v / np.sqrt(2))
    return np.maximum(v, 0.0) if act == "relu" else v


def epilogue(x, q, s, group, act="none", bias=None, residual=None, scale=1.0):
    """(y, bound). Every activation has slope at most 1.13. Its own error: the exponent
    (or erfc's argument, squared) is rounded a few times, which the exponential turns
    into as many half steps times its size, at most 2 v^2 + |v|^3 for |v| of the sizes
    here; exponential, quotient and products add well under 64. Results below the
    smallest normal number may be flushed."""
    scale = float(np.float32(scale))  # a float of the interface
    p, d = product(x, q, s, group)
    if bias is not None:
        p = p + bias
        d = d + F32 * (np.abs(p) + d)

    def act_of(v, dv):
        a = activation(v, act)
        if act == "none" or act == "relu":
            return a, dv
        w = np.abs(v) + dv
        return a, 1.13 * dv + (64 + 2 * w ** 2 + w ** 3) * F32 * np.abs(a) + 2.0 ** -126

    if act in ("swiglu", "geglu"):
        n = q.shape[0] // 2
        g, dg = act_of(p[:, :n], d[:, :n])
        u, du = p[:, n:], d[:, n:]
        y, d = g * u, dg * (np.abs(u) + du) + np.abs(g) * du
        d = d + F32 * (np.abs(y) + d)
    else:
        y, d = act_of(p, d)
    y, d = scale * y, abs(scale) * d
    d = d + F32 * (np.abs(y) + d)
    if residual is not None:
        y = y + residual
        d = d + F32 * (np.abs(y) + d)
    return y, d + BF16 * (np.abs(y) + d)


# Additions a sum of a row can pass through: 8 pieces of 8 in a thread, 6 steps in a
# wave, 16 waves.
STEPS = 8 * 8 + 6 + 16


def _normalise(v, dv, kind, eps, weight, bias, unit):
    """(norm of rows v known to within dv, bound). With m the mean, a deviation is off by
    dv, by the mean of dv, by the sum's STEPS + 2 half steps of the mean magnitude and by
    its own rounding; a root mean square of n values off by e moves by at most rms(e), and
    its sum, mean, root and quotient by STEPS / 2 + 6 half steps."""
    if kind == "layer":
        m = v.mean(1, keepdims=True)
        dm = dv.mean(1, keepdims=True) + (STEPS + 2) * F32 * (np.abs(v) + dv).mean(1, keepdims=True)
        v = v - m
        dv = dv + dm
        dv = dv + F32 * (np.abs(v) + dv)
    with np.errstate(divide="ignore"):
        r = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    dr = np.sqrt((dv * dv).mean(1, keepdims=True)) * r + (STEPS / 2 + 6) * F32  # relative
    w = np.ones(v.shape[1]) if weight is None else weight + (1.0 if unit else 0.0)
    x = v * r * w
    d = np.abs(w) * r * dv * (1 + dr) + (dr + 4 * F32) * np.abs(x)
    if bias is not None:
        x = x + bias
        d = d + F32 * (np.abs(x) + d)
    return x, d


def norm(y=None, residual=None, kind="rms", eps=1e-6, post=False, post_weight=None, post_bias=None,
         gate=None, gate_rows=1, scale=1.0, weight=None, bias=None, unit=False):
    """((r, bound), (v, bound)) before their last rounding."""
    scale, eps = float(np.float32(scale)), float(np.float32(eps))  # floats of the interface
    if y is not None:
        u, d = y, np.zeros_like(y)
        if post:
            u, d = _normalise(u, d, kind, eps, post_weight, post_bias, unit)
        if gate is not None:
            g = gate[np.arange(y.shape[0]) // gate_rows]
            u, d = u * g, d * np.abs(g)
            d = d + F32 * (np.abs(u) + d)
        u, d = scale * u, abs(scale) * d
        d = d + F32 * (np.abs(u) + d)
        r = u if residual is None else u + residual
        d = d + F32 * (np.abs(r) + d)
    else:
        r, d = residual, np.zeros_like(residual)
    return (r, d), _normalise(r, d, kind, eps, weight, bias, unit)


def codes(got_q, got_s, v, d):
    """Whether codes (natural order) and scales stand for rows v known to within d: the
    scale within the largest value's error and two roundings, each code's value within
    half a unit (its product rounded twice) of the value."""
    a = np.abs(v).max(1)
    ok = np.abs(got_s - a / 127) <= d.max(1) / 127 + 2 * F32 * a / 127
    unit = got_s[:, None].astype(np.float64)
    tol = 0.5 * unit + d + 127 * unit * 4 * F32 + 2 * F32 * np.abs(v)
    return ok.all() and bool(np.all(np.abs(got_q * unit - v) <= tol)) and np.abs(got_q).max() <= 127


def natural(c: np.ndarray) -> np.ndarray:
    """Stored order of w4a8_quantize -> natural order."""
    T, N = c.shape
    back = np.argsort(moe_ref.ORDER)
    return c.reshape(T, N // 16, 16)[:, :, back].reshape(T, N)


def moe_layer(x, logits, q_up, s_up, q_down, s_down, group, top_k, base=None, live=None,
              bias=None, **route):
    """x fp64 [T][H], logits fp64 [T][E] (their definition is the caller's), experts' codes
    and scales. Returns ids, weights, out, bound. h is off by its product's bound (that
    of moe_ref.experts without its last rounding) and held as two bf16: the second rounds
    a remainder of at most 2^-8 of it by 2^-8. down's biased sums run over both, and over
    the groups of all chosen experts, waves and parts: 2 group + top_k G + 44 half steps
    of their weighted magnitudes, and the weights' own rounding."""
    z = np.array(logits, np.float64)
    if live is not None:
        z[np.asarray(live) == 0] = -np.inf
    ids, w, off, rows = moe_ref.route(z, bias, top_k, **route)
    T, E = z.shape
    H, I = q_down.shape[1:]
    h, dh = moe_ref.experts(x, q_up, s_up, rows, off, top_k, group, True)
    dh = (dh - BF16 * np.abs(h)) / (1 + BF16)
    dh = dh + BF16 ** 2 * (np.abs(h) + dh)
    out = np.zeros((T, H)) if base is None else base.copy()
    d = np.zeros((T, H))
    for t in range(T):
        for j in range(top_k):
            e = ids[t, j]
            if e < 0:
                continue
            sl = t * top_k + j
            se = np.repeat(s_down[e], group, axis=1)
            wd = q_down[e] * se
            out[t] += w[t, j] * (wd @ h[sl])
            mag = ((np.abs(24.0 + q_down[e]) + 24.0) * np.abs(se)) @ ((1 + 2 * BF16) * np.abs(h[sl]) + dh[sl])
            d[t] += abs(w[t, j]) * (np.abs(wd) @ dh[sl]
                                    + (2 * group + top_k * (I // group) + 44) * F32 * mag)
    d = d + F32 * (np.abs(out) + d)
    return ids, w, out, d + BF16 * (np.abs(out) + d)
