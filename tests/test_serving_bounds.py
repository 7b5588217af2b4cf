"""The bounds that test_gpu_serving_long.py holds fp32 outputs to, against a
model of the kernel's arithmetic on the CPU: weights in three bf16 pieces and
sums that start again every 1024 tokens stay within them; two pieces, one, or
sums that never start again do not."""
import numpy as np
import pytest
import torch

from tests import serving_bounds as sb


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def _pieces(w, n):
    """Sum of the first n bf16 pieces of fp32 weights, each the rounding of
    what the ones before left."""
    total, rest = np.zeros(w.shape), w.astype(np.float32)
    for _ in range(n):
        p = _bf16(rest)
        total, rest = total + p, (rest - p).astype(np.float32)
    return total


def _exact(q, K, V, scale2):
    return sb.exact(*(torch.from_numpy(np.asarray(x, dtype=np.float64)) for x in (q, K, V)), scale2)


@pytest.mark.parametrize("pieces", [1, 2, 3])
def test_weights_in_pieces(pieces):
    sm = 0.0731
    scale2 = sb.scale2_of(sm)
    q, K, V = sb.two_tokens(200, 64, 1)
    e = _exact(q, K, V, scale2)
    # fp32 as in the kernel: the reference is the larger score, the exponential rounded to nearest
    x = (q.astype(np.float64) @ K.T).astype(np.float32) * np.float32(scale2)
    w = np.exp2((x - x.max(-1, keepdims=True)).astype(np.float64)).astype(np.float32)
    out = (_pieces(w, pieces) @ V / w.sum(-1, dtype=np.float32)[:, None]).astype(np.float32)
    tol, _ = sb.bounds(e, True, 1)
    over = np.abs(out - e["out"].numpy()) > tol.numpy()
    assert not over.any() if pieces == 3 else over.mean() > 0.1


def _towards_zero(x):
    """fp64 to 24 significant bits, towards zero."""
    f, ex = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(f, 24)), ex - 24)


@pytest.mark.parametrize("period", [sb.PERIOD, 1 << 30])
def test_sums_that_start_again(period):
    tiles, d = 256, 8
    K, V = sb.long_sums(tiles * sb.TILE, d, 2)
    q = np.zeros((1, d))
    q[0, 0] = 1.0
    assert sb.scale2_of(sb.LN2_SCALE) == 1.0
    e = _exact(q, K, V, 1.0)
    w = np.exp2(K[:, 0].astype(np.float64))
    steps = (w[:, None] * V).reshape(-1, 16, d).sum(1)              # exact
    total, acc = np.zeros(d, dtype=np.float32), np.zeros(d)
    for i, s in enumerate(steps):
        if i % (period * 8) == 0:
            total, acc = (total + acc).astype(np.float32), np.zeros(d)
        acc = _towards_zero(acc + s)
    out = (total + acc.astype(np.float32)) / np.float32(w.sum())
    tol, _ = sb.bounds(e, True, tiles, exact_sums=True)
    over = np.abs(out - e["out"].numpy()) > tol.numpy()
    assert over.mean() > 0.5 if period > tiles else not over.any()
