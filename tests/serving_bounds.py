"""Exact attention values and error bounds for the tests of mxs_attn_tree over
many tiles, and the inputs of the two tests that a lower precision must fail.

A score is an exact fp32 number here: queries are multiples of 1/2 below 32
and keys multiples of 2^-8, so that every partial sum of products has fewer
than 24 bits.  What is left, in units u = 2^-24 of S = sum_p w_p |V_p| (w the
softmax weights) unless stated otherwise:

  a score in base 2, x = s * scale, rounded, and its difference from the
    reference, rounded: u (|x| + |x - ref|) absolute, ln 2 times that in the
    weight; |x - ref| is at most the range of the row's scores;
  the exponential: 2^-22 relative;
  the weight as it enters the product with V: three bf16 pieces, u, for an
    fp32 output; one, 2^-8, for bf16;
  the tensor core's sums: rounded towards zero, at most 2 u of the sum for
    each 16 tokens; an fp32 output's start again after 1024 tokens;
  the sums taken outside: one rounding, u, for each addition;
  a reference that moved (scores that range over more than 2^24): the factor
    2^(old - new) with an argument of at most 24 that matters, and its product;
  parts of several CTAs: the logarithm of a part's sum (one unit of a value
    below 41), less its reference, rounded, and the difference from the
    largest; 2^() of it; one rounding for each part;
  absolute: weights below 2^-126 of the largest are zero.  Where all others
    meet a V of zero they are the whole result: n 2^-126 max|V|, less than
    2^-100 for up to 2^20 tokens and values below 2^6.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24
LN2 = math.log(2.0)
TILE, PERIOD = 128, 8


def scale2_of(sm_scale: float) -> float:
    """The factor of scores in base 2 as the call takes it: fp32."""
    return float(np.float32(float(np.float32(sm_scale)) * 1.4426950408889634))


def exact(q, K, V, scale2, see=None):
    """Rows q (n, d) over tokens K, V (t, d), all fp64: a dict of out, lse
    (base 2), S, and each row's range and largest magnitude of its scores."""
    x = (q @ K.T) * scale2
    hidden = torch.zeros_like(x, dtype=torch.bool) if see is None else ~see
    top = x.masked_fill(hidden, -math.inf).amax(-1)
    low = x.masked_fill(hidden, math.inf).amin(-1)
    w = torch.exp2((x - top[:, None]).masked_fill(hidden, -math.inf))
    l = w.sum(-1)
    return dict(out=(w @ V) / l[:, None], S=(w @ V.abs()) / l[:, None], lse=top + torch.log2(l), range=top - low,
                size=torch.maximum(top.abs(), low.abs()))


def bounds(e, fp32, tiles, joined=0, wide=False, exact_sums=False):
    """(of the output, of the natural lse) for rows of exact(), where a CTA
    has up to `tiles` tiles of an item in turn and an item up to `joined` CTAs
    (0: none is joined).  exact_sums: the weights are powers of two whose sum
    is an fp32 number."""
    r, big = e["range"], e["size"]
    score = LN2 * (big + r) * U + 4 * U
    moved = torch.where(r > 24, torch.full_like(r, 2 * (4 + 24 * LN2 + 2) * U), torch.zeros_like(r))
    adds = 0 if exact_sums else (32 if wide else 1) * tiles + 7
    total = score + moved / 2 + adds * U
    steps = min(tiles, PERIOD) if fp32 else tiles
    rel = score + (U if fp32 else 2.0 ** -8) + moved / 2 + steps * (TILE // 16) * 2 * U + (tiles / PERIOD + 3) * U
    rel = rel + total + 2 * U
    part = LN2 * (2 * 41 + big + 17 + 24) * U
    if joined > 1:
        rel = rel + 2 * (part + 4 * U) + (2 * joined + 3) * U
        total = total + part + 4 * U + joined * U
    out = 2.0 ** -100 + rel[:, None] * e["S"] + (U if fp32 else 2.0 ** -8) * e["out"].abs()
    return out, total + LN2 * (2 * 41 + 17 + 3 * big) * U + 3 * U * LN2 * e["lse"].abs()


def columns(fp32, max_q, rep, d, bits):
    """Columns of a row tile (256: the wide form)."""
    rows, most = max_q * rep, 32 if fp32 and d == 128 and bits == 8 else 64
    return 16 if rows <= 16 else 32 if rows <= 32 else most if rows <= 64 or fp32 else 256


def cut(ctx, counts, rep, n_kvh, R, causal, max_q, ctas):
    """How the call is cut: (most tiles of one item in turn in a CTA, most
    CTAs of an item, most items of a CTA, CTAs that go from items of one half
    to items of two)."""
    items = []
    for a, n in zip(ctx, counts):
        for rt in range(-(-max_q * rep // R)):
            if rt * R >= n * rep:
                continue
            total = a + (min(n, (rt * R + R - 1) // rep + 1) if causal else n)
            items += [(-(-total // TILE), n * rep - rt * R > 128)] * n_kvh
    total = sum(t for t, _ in items)
    ctas = min(ctas, total)
    size, more = divmod(total, ctas)
    run, spread, most, turns = 0, 0, 0, 0
    at, i, used, parts = 0, 0, 0, [0] * len(items)
    for c in range(ctas):
        left, mine, halves = size + (c < more), 0, []
        while left > 0:
            n = min(left, items[i][0] - used)
            run, mine = max(run, n), mine + 1
            halves.append(items[i][1])
            parts[i] += 1
            used += n
            left -= n
            if used == items[i][0]:
                i, used = i + 1, 0
        most = max(most, mine)
        turns += any(b and not a for a, b in zip(halves, halves[1:]))
    return run, max(parts), most, turns


# ------------------------------------------- inputs that a lower precision fails
def two_tokens(n, d, seed):
    """Two tokens for each of n rows: one with the largest score and V = 0,
    the other with a weight below 1 of many bits: out = w V / (1 + w), where
    S = |out|, so that the error is that of w alone."""
    rng = np.random.default_rng(seed)
    q = np.zeros((n, d), dtype=np.float32)
    q[:, 0] = np.arange(1, n + 1) % 64 * 0.5                       # exact in bf16
    K = np.zeros((2, d), dtype=np.float32)
    K[0, 0] = 1.0
    V = np.zeros((2, d), dtype=np.float32)
    V[1] = (rng.integers(64, 128, d) / 64.0) * np.where(rng.random(d) < 0.5, -1.0, 1.0)
    return q, K, V


def long_sums(tokens, d, seed):
    """Positive values of several magnitudes: sums that grow by every token,
    whose rounding towards zero adds up.  Scores are integers from -3 to 0 in
    base 2, so that weights are powers of two and their sum has few bits."""
    rng = np.random.default_rng(seed)
    K = np.zeros((tokens, d), dtype=np.float32)
    K[:, 0] = -rng.integers(0, 4, tokens).astype(np.float32)
    K[0, 0] = 0.0
    V = (rng.integers(64, 128, (tokens, d)) / 128.0 * 2.0 ** -rng.integers(0, 4, (tokens, 1))).astype(np.float32)
    return K, V


LN2_SCALE = float(np.float32(LN2))                                  # scale2_of: 1
