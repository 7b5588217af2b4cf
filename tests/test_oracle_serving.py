"""Pins for the fp64 references of the serving operators (rotary positions,
attention of drafted tokens), by routes that share nothing with them."""
import cmath
import math

import numpy as np
import pytest

from oracle import serving

YARN = dict(kind="yarn", factor=16.0, orig_len=8192, beta_fast=32.0, beta_slow=1.0)
PARTS = dict(kind="parts", factor=8.0, low=1.0, high=4.0, orig_len=8192)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_a_complex_product(layout):
    rng = np.random.default_rng(0)
    x, pos = rng.normal(size=(3, 2, 12)), [0, 5, -7]
    y = serving.rope(x, pos, 8, 100.0, layout)
    for t in range(3):
        for i in range(4):
            u, v = (i, i + 4) if layout == "half" else (2 * i, 2 * i + 1)
            z = (x[t, :, u] + 1j * x[t, :, v]) * cmath.exp(1j * pos[t] * 100.0 ** (-i / 4))
            assert np.allclose(y[t, :, u], z.real, atol=1e-14) and np.allclose(y[t, :, v], z.imag, atol=1e-14)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])


@pytest.mark.parametrize("scaling", [None, dict(kind="linear", factor=4.0), PARTS, YARN])
def test_rope_inverse_is_the_transpose(scaling):
    rng = np.random.default_rng(1)
    x, g, pos = rng.normal(size=(4, 2, 16)), rng.normal(size=(4, 2, 16)), [3, 100, 5000, 12345]
    y = serving.rope(x, pos, 16, 5e5, "half", scaling)
    back = serving.rope(g, pos, 16, 5e5, "half", scaling, inverse=True)
    assert math.isclose((y * g).sum(), (x * back).sum(), rel_tol=1e-12)


def test_rope_scaling_ends():
    """Fast pairs keep their frequency, slow ones are divided by the factor,
    as long as the blend's borders say so."""
    plain, _ = serving.rope_frequencies(128, 5e5)
    for sc in (PARTS, YARN):
        f, gain = serving.rope_frequencies(128, 5e5, sc)
        assert f[0] == plain[0] and f[-1] == plain[-1] / np.longdouble(sc["factor"])
        assert all(a >= b for a, b in zip(f, f[1:]))
        assert gain == (1.0 if sc is PARTS else 0.1 * math.log(16.0) + 1.0)
    # parts: a pair with t turns over the original length, low < t < high
    t = 8192 * plain / (2 * np.pi)
    i = next(j for j in range(64) if 1 < t[j] < 4)
    keep = (t[i] - 1) / 3
    f, _ = serving.rope_frequencies(128, 5e5, PARTS)
    assert math.isclose(f[i], plain[i] * keep + plain[i] / 8 * (1 - keep), rel_tol=1e-12)


def test_attention_two_tokens_and_masks():
    k = np.zeros((8, 1, 32))
    v = np.arange(8.0)[:, None, None] * np.ones((8, 1, 32))
    k[6, 0, 0] = math.log(3.0)
    q = np.zeros((3, 1, 32))
    q[:, 0, 0] = 1.0
    # one context token in slot 6 (page 3 of size 2), drafted tokens in slots 7, 0, 1
    pages = [[3, 0]]
    mask = np.array([[0], [0b010], [0b101]], dtype=np.uint32)
    out, lse, _ = serving.attn_tree(q, k, v, [0, 3], [1], pages, 2, 1.0, mask)
    assert np.allclose(out[0], 6.0) and math.isclose(lse[0, 0], math.log(3.0))
    assert np.allclose(out[1], (3 * 6 + 0) / 4) and math.isclose(lse[1, 0], math.log(4.0))
    assert np.allclose(out[2], (3 * 6 + 7 + 1) / 5)
    chain, _, _ = serving.attn_tree(q, k, v, [0, 3], [1], pages, 2, 1.0)
    assert np.allclose(chain[1], (3 * 6 + 7 + 0) / 5)


def test_attention_empty_row_and_rows_of_no_sequence():
    q, k = np.ones((4, 2, 32)), np.ones((2, 1, 32))
    out, lse, _ = serving.attn_tree(q, k, k, [1, 3], [0], [[0, 1]], 1, 1.0, np.zeros((4, 1), np.uint32))
    assert np.all(out[1:3] == 0) and np.all(np.isneginf(lse[1:3]))
    assert np.all(np.isnan(out[0])) and np.all(np.isnan(out[3]))
