"""mxs_attn_tree where a CTA goes through many tiles: references that move
under sums already taken, output periods that end, stages that are used again,
further items with another query, and turns from one half of the wide form to
two.  Queries are multiples of 1/2, so scores are exact and the bounds of
serving_bounds.py are close to what the kernels do; each test asserts how many
tiles of an item a CTA has in turn."""
import math

import numpy as np
import pytest
import torch

from tests import parity
from tests import serving_bounds as sb
from tests.test_gpu_serving import _trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c():
    parity.need_gpu()
    return parity.capi()


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _batch(c, ctx, counts, n_qh, n_kvh, d, bits, page, causal, seed, ramp=None):
    """A ragged batch over randomly placed pages.  ramp(positions): added to
    the first value of the keys there."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, max_len = len(ctx), max(a + b for a, b in zip(ctx, counts))
    per = -(-max_len // page)
    pages = torch.from_numpy(rng.permutation(B * per + 2)[: B * per].reshape(B, per).astype(np.int32)).cuda()
    cache = c.kv_cache_empty((B * per + 2) * page, n_kvh, d, bits)
    slots = []
    for b in range(B):
        p = torch.arange(ctx[b] + counts[b], device="cuda")
        slots.append(pages[b].long()[p // page] * page + p % page)
        k, v = (torch.randn((p.numel(), n_kvh, d), generator=g, device="cuda") for _ in range(2))
        if ramp is not None:
            k[:, :, 0] = ramp(p.float())[:, None]
        c.mxs_kv_write(k, v, cache, slots[-1])
    rows = sum(counts)
    q = ((torch.randn((rows, n_qh, d), generator=g, device="cuda") * 2).round() / 2).to(torch.bfloat16)
    words = -(-max(counts) // 32)
    mask = None if causal else torch.from_numpy(_trees(counts, words, seed).view(np.int32)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    qs = [sum(counts[:b]) for b in range(B + 1)]
    batch = c.tree_batch(torch.tensor(qs, **i32), torch.tensor(ctx, **i32), pages, page, max_q=max(counts), max_len=max_len,
                         mask=mask)
    return q, cache, batch, slots, qs, mask


def _check(c, q, cache, slots, qs, ctx, counts, mask, sm, dtype, got, lse, tiles, joined, wide=False):
    fp32, scale2 = dtype == torch.float32, sb.scale2_of(sm)
    n_qh, n_kvh = q.shape[1], cache.n_kvh
    rep, worst = n_qh // n_kvh, 0.0
    for b, n in enumerate(counts):
        if n == 0:
            continue
        K, V = c.mxs_kv_read(cache, slots[b], dtype=torch.float32)
        total = ctx[b] + n
        see = torch.ones((n, total), dtype=torch.bool, device="cuda")
        if mask is None:
            see[:, ctx[b]:] = torch.ones((n, n), device="cuda").tril() > 0
        else:
            m, j = mask[qs[b]: qs[b] + n].long(), torch.arange(n, device="cuda")
            see[:, ctx[b]:] = (m[:, j // 32] >> (j % 32)) & 1 > 0
        for g in range(n_kvh):
            at = (slice(qs[b], qs[b] + n), slice(g * rep, (g + 1) * rep))
            e = sb.exact(q[at].double().reshape(n * rep, -1), K[:, g].double(), V[:, g].double(), scale2,
                         see.repeat_interleave(rep, 0))
            tol, tol_lse = sb.bounds(e, fp32, tiles, joined, wide)
            off = (got[at].double().reshape(n * rep, -1) - e["out"]).abs()
            assert bool((off <= tol).all()), (b, g, (off / tol).max().item())
            worst = max(worst, (off / tol).max().item())
            off = (lse[at].double().reshape(-1) - e["lse"] * math.log(2.0)).abs()
            assert bool((off <= tol_lse).all()), (b, g, (off / tol_lse).max().item())
    return worst


def _run(c, shape, dtype, sm, seed, least, ramp=None, q_first=None, turns=0):
    ctx, counts, n_qh, n_kvh, d, bits, page, causal = shape
    q, cache, batch, slots, qs, mask = _batch(c, *shape, seed, ramp)
    if q_first is not None:
        q[:, :, 0] = q_first(torch.arange(q.shape[0] * n_qh, device="cuda")).view(q.shape[0], n_qh).to(torch.bfloat16)
    rep, fp32 = n_qh // n_kvh, dtype == torch.float32
    R = sb.columns(fp32, max(counts), rep, d, bits)
    run, parts, items, turned = sb.cut(ctx, counts, rep, n_kvh, R, causal, max(counts), _sms())
    assert run >= least and turned >= turns
    out, lse = c.mxs_attn_tree(q, cache, batch, sm, dtype=dtype, return_lse=True)
    c.mxs_sync()
    _check(c, q, cache, slots, qs, ctx, counts, mask, sm, dtype, out, lse, run, parts, R == 256)
    assert torch.equal(c.mxs_attn_tree(q, cache, batch, sm, dtype=dtype), out)
    return R


LONG = [
    # ctx, counts, n_qh, n_kvh, d, bits, page, causal
    ([20000, 16000, 14000], [2, 1, 2], 32, 8, 128, 4, 64, True),               # 16 columns
    ([16000, 9000, 12000, 14000], [7, 5, 3, 7], 24, 8, 64, 8, 33, False),      # 32
    ([15000, 13000, 12001], [16, 9, 12], 32, 8, 128, 4, 16, False),            # 64
    ([14000, 15000], [16, 15], 32, 8, 128, 8, 128, False),                     # 64; of 32 in two row tiles for fp32
    ([15000, 12000], [64, 40], 32, 8, 128, 4, 64, False),                      # the wide form, two halves; 64
    ([9000, 7000, 8000], [50, 75, 20], 64, 8, 64, 8, 16, True),                # several row tiles, the last of one half
]
KINDS = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", KINDS, ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", LONG, ids=[str(i) for i in range(len(LONG))])
def test_many_tiles_in_turn(c, shape, dtype):
    _run(c, shape, dtype, 0.04, 100, sb.PERIOD + 2)


@pytest.mark.parametrize("dtype", KINDS, ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("counts,n_qh", [([3, 2], 32), ([16, 9], 32), ([64, 30], 32)])   # 16 and 64 columns, the wide form
def test_references_that_move_in_turn(c, counts, n_qh, d, dtype):
    """Scores that rise by some 60 (base 2) within a CTA's tiles for some
    heads, fall for others: references move at t > 0 and between the ends of
    output periods, while other columns' stay."""
    first = lambda i: (i % 7 - 3.0) * 5.0                          # -15 .. 15
    shape = ([20000, 18000], counts, n_qh, 8, d, 8, 16, False)
    _run(c, shape, dtype, 0.25, 200, sb.PERIOD + 2, ramp=lambda p: (p * 0.004).floor(), q_first=first)


@pytest.mark.parametrize("dtype", KINDS, ids=["bf16", "fp32"])
@pytest.mark.parametrize("n_qh", [32, 8])
def test_a_step_far_above_late_in_an_item(c, n_qh, dtype):
    """One token late in each item far above all before it: by more than
    2^24, and by so much that everything before is lost."""
    first = lambda i: torch.tensor([8.0, 1.0, -2.0, 0.0], device="cuda")[i % 4]
    for top in (60.0, 1000.0):
        shape = ([19999, 17003], [9, 16], n_qh, 8, 128, 8, 64, True)
        _run(c, shape, dtype, 0.25, 300, sb.PERIOD + 2, ramp=lambda p: (p % 6007 == 6000) * top, q_first=first)


@pytest.mark.parametrize("dtype", KINDS, ids=["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
def test_items_of_one_half_and_of_two_in_turn(c, causal, dtype):
    """Short items, several to a CTA, whose queries fill one half of the wide
    form or both; lengths that end inside a tile, at its border and behind it."""
    rng = np.random.default_rng(7)
    counts = [int(n) for n in rng.integers(1, 76, 60)]
    ctx = [int(n) for n in rng.integers(0, 900, 60)]
    ctx[:3], counts[:3] = [128 - 20, 128 - 33, 1024 - 70], [20, 34, 70]
    R = _run(c, (ctx, counts, 32, 8, 64, 4, 16, causal), dtype, 0.09, 400, 2, turns=10 if dtype == torch.bfloat16 else 0)
    assert R == (256 if dtype == torch.bfloat16 else 64)


@pytest.mark.parametrize("counts,n_qh", [([1] * 90, 16), ([7] * 90, 32), ([16] * 90, 32)])
@pytest.mark.parametrize("dtype", KINDS, ids=["bf16", "fp32"])
def test_short_items_in_turn(c, counts, n_qh, dtype):
    rng = np.random.default_rng(8)
    ctx = [int(n) for n in rng.integers(0, 700, len(counts))]
    _run(c, (ctx, counts, n_qh, 8, 128, 8, 5, True), dtype, 0.05, 500, 3)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rep", [4, 20, 64])                         # 16, 32 and 64 columns
def test_weights_of_an_fp32_output_have_24_bits(c, rep, d, bits):
    """Fails with weights of two bf16 pieces, as test_serving_bounds.py shows."""
    sm, B = 0.0731, 50
    q, K, V = sb.two_tokens(B * rep, d, 1)
    cache = c.kv_cache_empty(2, 1, d, bits)
    k, v = (torch.from_numpy(x).cuda()[:, None, :] for x in (K, V))
    c.mxs_kv_write(k, v, cache, torch.arange(2, device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = c.tree_batch(torch.arange(B + 1, **i32), torch.ones(B, **i32), torch.zeros((B, 1), **i32), 2, max_q=1, max_len=2)
    qt = torch.from_numpy(q).cuda().view(B, rep, d).to(torch.bfloat16)
    out, lse = c.mxs_attn_tree(qt, cache, batch, sm, dtype=torch.float32, return_lse=True)
    c.mxs_sync()
    K, V = (x[:, 0].double() for x in c.mxs_kv_read(cache, torch.arange(2, device="cuda"), dtype=torch.float32))
    e = sb.exact(qt.double().reshape(-1, d), K, V, sb.scale2_of(sm))
    tol, tol_lse = sb.bounds(e, True, 1)
    assert bool(((out.double().reshape(-1, d) - e["out"]).abs() <= tol).all())
    assert bool(((lse.double().reshape(-1) - e["lse"] * math.log(2.0)).abs() <= tol_lse).all())


@pytest.mark.parametrize("bits,d", [(8, 64), (8, 128), (4, 64)])
@pytest.mark.parametrize("rep", [4, 20, 40])                         # 16, 32 and 64 columns
def test_sums_of_an_fp32_output_start_again(c, rep, d, bits):
    """256 tiles of an item in each CTA.  Fails with sums that stay in the
    tensor core, as test_serving_bounds.py shows."""
    tiles, B = 256, _sms()
    n = tiles * sb.TILE
    K, V = sb.long_sums(n, d, 2)
    cache = c.kv_cache_empty(n, 1, d, bits)
    k, v = (torch.from_numpy(x).cuda()[:, None, :] for x in (K, V))
    c.mxs_kv_write(k, v, cache, torch.arange(n, device="cuda"))
    q = torch.zeros((B, rep, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = torch.arange(rep, device="cuda") % 3
    i32 = dict(dtype=torch.int32, device="cuda")
    # (every sequence over the same pages: one item for each CTA)
    batch = c.tree_batch(torch.arange(B + 1, **i32), torch.full((B,), n - 1, **i32), torch.zeros((B, 1), **i32), n, max_q=1,
                         max_len=n)
    wide = 2 if rep == 40 and d == 128 and bits == 8 else 1             # (32 columns there: two row tiles)
    assert sb.cut([n - 1] * B, [1] * B, rep, 1, sb.columns(True, 1, rep, d, bits), True, 1, _sms())[:3] == (tiles, 1, wide)
    out = c.mxs_attn_tree(q, cache, batch, sb.LN2_SCALE, dtype=torch.float32)
    c.mxs_sync()
    K, V = (x[:, 0].double() for x in c.mxs_kv_read(cache, torch.arange(n, device="cuda"), dtype=torch.float32))
    e = sb.exact(q[0].double(), K, V, 1.0)
    tol, _ = sb.bounds(e, True, tiles, exact_sums=True)
    assert bool(((out.double() - e["out"]).abs() <= tol).all())
