"""fp64 references of the serving operators: rotary positions, and attention of
drafted tokens over a paged K/V cache.  Test infrastructure only; plain numpy,
one token and one head at a time, sharing nothing with the CUDA path.

The pages keep the K/V cache in MXINT blocks ([TS §4] W4A4KV4); the rotary and
attention formulas are the textbook ones, stated at each function.
"""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot: int, theta: float, scaling=None):
    """(long double angle per position of each pair, factor of cos and sin)."""
    L = np.longdouble
    two_pi = L(2) * L("3.14159265358979323846264338327950288")
    freqs, gain = [], 1.0
    for i in range(rot // 2):
        w = L(theta) ** (L(-2 * i) / L(rot))
        if scaling is None:
            freqs.append(w)
            continue
        factor = L(scaling["factor"])
        if scaling["kind"] == "linear":
            freqs.append(w / factor)
            continue
        turns = L(scaling["orig_len"]) * w / two_pi            # turns over the original length
        if scaling["kind"] == "parts":
            keep = (turns - L(scaling["low"])) / (L(scaling["high"]) - L(scaling["low"]))
        else:
            def place(n):
                return L(rot) * np.log(L(scaling["orig_len"]) / (two_pi * L(n))) / (L(2) * np.log(L(theta)))
            a = max(L(0), np.floor(place(scaling.get("beta_fast", 32.0))))
            b = min(L(rot - 1), np.ceil(place(scaling.get("beta_slow", 1.0))))
            keep = L(1) - min(L(1), max(L(0), (L(i) - a) / max(L("0.001"), b - a)))
            gain = 0.1 * math.log(float(factor)) + 1.0
        keep = min(L(1), max(L(0), keep))
        freqs.append(w * (keep + (L(1) - keep) / factor))
    return np.array(freqs, dtype=np.longdouble), gain


def rope(x, pos, rot: int, theta: float, layout: str = "half", scaling=None, inverse: bool = False) -> np.ndarray:
    """x (tokens, heads, d) fp64 with the first `rot` positions of each head
    turned in pairs: (u, v) -> (u cos a - v sin a, v cos a + u sin a)."""
    x = np.asarray(x, dtype=np.float64)
    f, gain = rope_frequencies(rot, theta, scaling)
    y = x.copy()
    for t in range(x.shape[0]):
        angle = np.longdouble(int(pos[t])) * f
        c, s = (np.cos(angle) * gain).astype(np.float64), (np.sin(angle) * gain).astype(np.float64)
        if inverse:
            s = -s
        for i in range(rot // 2):
            u, v = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            y[t, :, u] = x[t, :, u] * c[i] - x[t, :, v] * s[i]
            y[t, :, v] = x[t, :, v] * c[i] + x[t, :, u] * s[i]
    return y


def attn_tree(q, k, v, q_start, length, pages, page_size: int, sm_scale: float, mask=None):
    """(out, lse, spread) in fp64.  q (rows, n_qh, d); k, v: decoded cache
    (n_slots, n_kvh, d); mask (rows, words) uint32 or None for a chain.
    spread[r, h] = the largest sum_e |q_e k_pe| over the tokens seen, for
    error bounds.  Rows of no sequence hold NaN."""
    rows, n_qh, d = q.shape
    rep = n_qh // k.shape[1]
    out, lse = np.full((rows, n_qh, d), np.nan), np.full((rows, n_qh), np.nan)
    spread = np.zeros((rows, n_qh))
    for b in range(len(length)):
        ctx, n = int(length[b]), int(q_start[b + 1] - q_start[b])
        p = np.arange(ctx + n)
        slots = np.asarray(pages[b], dtype=np.int64)[p // page_size] * page_size + p % page_size
        for i in range(n):
            r = int(q_start[b]) + i
            if mask is None:
                sees = p <= ctx + i
            else:
                sees = np.array([t < ctx or bool((int(mask[r][(t - ctx) // 32]) >> ((t - ctx) % 32)) & 1) for t in p],
                                dtype=bool)
            at = slots[sees]
            for h in range(n_qh):
                kk, vv = k[at, h // rep], v[at, h // rep]
                if at.size == 0:
                    out[r, h], lse[r, h] = 0.0, -np.inf
                    continue
                s = sm_scale * (kk @ q[r, h])
                m = s.max()
                e = np.exp(s - m)
                out[r, h], lse[r, h] = (e @ vv) / e.sum(), m + np.log(e.sum())
                spread[r, h] = (np.abs(kk) @ np.abs(q[r, h])).max()
    return out, lse, spread
