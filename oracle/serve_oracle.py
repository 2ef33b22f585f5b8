"""fp64 CPU oracle of the serving operators: the cache append with its norms and
rotation, paged attention, and sampling. Plain numpy loops from the
definitions in include/q4dec_serve.h; shares no code with the HIP path."""
from __future__ import annotations

import numpy as np


def bf16_round(x):
    """Round to nearest even to bf16, as float64 (finite input)."""
    f = np.asarray(x, dtype=np.float64).astype(np.float32)
    b = f.view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def e4m3_values():
    """The 256 values of OCP e4m3 by their bits (0x7F and 0xFF are NaN)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        out[b] = np.nan if (b & 0x7F) == 0x7F else (-v if b & 0x80 else v)
    return out


def rope_row(x, position, freqs, half):
    """The pairs (j, j + half), j < len(freqs), of each head of x [heads, D] turned by position * freqs[j]."""
    x = np.array(x, dtype=np.float64)
    n = len(freqs)
    # in long double: an fp64 product at position 2^31 would keep only 22 fractional bits of the angle
    a = np.longdouble(int(position)) * np.asarray(freqs, dtype=np.longdouble)
    c, s = np.cos(a).astype(np.float64), np.sin(a).astype(np.float64)
    lo, hi = x[:, :n].copy(), x[:, half:half + n].copy()
    x[:, :n], x[:, half:half + n] = lo * c - hi * s, hi * c + lo * s
    return x


def rms_row(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x if weight is None else x * np.asarray(weight, dtype=np.float64)


def append(q, k, v, positions, freqs, half, q_norm=None, k_norm=None, v_norm=False, eps=1e-6):
    """Exact q, k, v rows [T, heads, D] before any rounding (None for a missing input)."""
    def one(x, norm, do_norm, turn):
        if x is None:
            return None
        rows = []
        for t in range(x.shape[0]):
            r = np.asarray(x[t], dtype=np.float64)
            if do_norm:
                r = rms_row(r, norm, eps)
            rows.append(rope_row(r, positions[t], freqs, half) if turn else r)
        return np.array(rows).reshape(x.shape)

    return (one(q, q_norm, q_norm is not None, True), one(k, k_norm, k_norm is not None, True),
            one(v, None, v_norm, False))


def attention(q, keys, values, q_lens, kv_lens, scale, window):
    """q: [T, Hq, D]; keys / values: per sequence [kv_len, Hkv, D] (fp64 values as stored).
    Returns (out [T, Hq, D], mag, span): mag = sum_j p_j |v_j|, span [T, Hq] = the largest
    |scale| * sum_d |q_d k_jd| over the positions a row sees. All zero for a row that sees nothing."""
    T, Hq, D = q.shape
    out, mag, span = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    t = 0
    for b, (n, long) in enumerate(zip(q_lens, kv_lens)):
        K, V = keys[b], values[b]
        g = Hq // K.shape[1]
        for i in range(n):
            p = long - n + i
            lo = max(0, p - window + 1) if window else 0
            if p >= 0:
                for h in range(Hq):
                    k, v = K[lo:p + 1, h // g], V[lo:p + 1, h // g]
                    s = scale * (k @ q[t, h])
                    w = np.exp(s - s.max())
                    w = w / w.sum()
                    out[t, h], mag[t, h] = w @ v, w @ np.abs(v)
                    span[t, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, h])).max()
            t += 1
    return out, mag, span


def attention_tolerance(out, mag, span, keys, dim):
    """Bound on |kernel - out|, from the roundings of the definition.

    A score is a sum of `dim` exact products in fp32, scaled and brought to base 2 (4 more roundings):
    off by at most ds = (dim + 4) 2^-24 span. A probability is then off by a factor of at most 1 + 1.1 ds
    + 2^-21 (the exponential) in the sum of weights, and by another half step of bf16, 2^-8, in the
    weighted sum; both sums add `keys` terms in fp32. The quotient of the two is rounded once to bf16."""
    ds = (dim + 4) * 2.0 ** -24 * span[..., None]
    rel = 2 * (1.1 * ds + 2.0 ** -21 + (keys + 8) * 2.0 ** -24) + 2.0 ** -8
    inner = mag * rel
    return inner + 2.0 ** -8 * (np.abs(out) + inner) + 1e-30


def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, cap=30.0):
    """(index, probability, border) of one row; border: the distance, as a share of the whole, from the
    drawn number or the top-p border to the nearest running sum it is compared with (1 where none is)."""
    z = np.asarray(z, dtype=np.float64)
    live = np.nonzero(z > -np.inf)[0]
    if not live.size:
        return -1, np.nan, 1.0
    order = live[np.argsort(-z[live], kind="stable")]
    if not temperature > 0:
        return int(order[0]), 1.0, 1.0
    x = (cap * np.tanh(z[order] / cap) if cap > 0 else z[order])
    w = np.where(z[order] == z[order[0]], 1.0, np.exp((x - x[0]) / temperature)) if np.isfinite(x[0]) else \
        (z[order] == z[order[0]]).astype(np.float64)
    border = 1.0
    if 0 < top_k < len(z):
        order, w = order[:top_k], w[:top_k]
    stay = np.ones(len(w), bool)
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        stay = before < top_p * w.sum()
        border = min(border, np.abs(before[1:] - top_p * w.sum()).min() / w.sum() if len(w) > 1 else 1.0)
    if min_p > 0:
        stay &= w >= min(min_p, 1.0)
    stay[0] = True
    order, w = order[stay], w[stay]
    by = np.argsort(order)
    order, w = order[by], w[by]
    run = np.cumsum(w)
    u = float(u) if u > 0 else 0.0
    at = min(int(np.searchsorted(run, min(u, 1.0) * run[-1], side="right")), len(w) - 1)
    if u < 1:
        border = min(border, np.abs(run - u * run[-1])[:-1].min() / run[-1] if len(w) > 1 else 1.0)
    return int(order[at]), w[at] / run[-1], border
