"""GPU parity of the serving operators: rotary positions, the K/V cache's
write and read, and attention of drafted tokens, against fp64 references.

Tolerances, derived:
  rope: the rotation is exact to far below fp32 (64-bit cos, sin, products),
    so the result is off by its roundings: 2^-24 relative to fp32, 2^-8 more
    for bf16 (half a step of 8 significant bits), plus 2^-40 of the pair's
    magnitude for the 64-bit evaluation (its error is some 2^-52).
  cache: codes and scales are equal bit for bit, the read values exactly.
  attention: decoded values are exact.  A score accumulates d exact products
    in fp32 in any order: off by at most d 2^-24 sum|q k| sm_scale, plus
    2^-23 |s| for the scaling in base 2, the subtraction of the maximum and
    the argument's rounding each (|s| <= sum|q k| sm_scale).  Both numerator
    and denominator carry that relative error, exp2's 2^-22 and the fp32
    sums' n 2^-24 over n tokens: 2 (ds + 2^-22 + n 2^-24).  The weights are
    rounded to 8 significant bits (2^-8) for a bf16 output and to 16 (2^-16)
    for fp32; the output is a convex combination, so all of it counts
    against max|V|.  The output's own rounding: 2^-8 or 2^-24 relative.
    lse: ds, and the sum's relative error, 2^-22 + n 2^-24, and 2^-23 |lse|
    for its own arithmetic.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving
from tests import parity

pytestmark = pytest.mark.gpu

PARTS = dict(kind="parts", factor=8.0, low=1.0, high=4.0, orig_len=8192)
YARN = dict(kind="yarn", factor=16.0, orig_len=8192)


@pytest.fixture(scope="module")
def c():
    parity.need_gpu()
    return parity.capi()


def _randn(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


# -------------------------------------------------------------------- rope
def _rope_bound(x, ref, bf16):
    m = np.abs(x).max(axis=-1, keepdims=True) * 2
    return np.abs(ref) * (2.0 ** -24 + (2.0 ** -8 if bf16 else 0.0)) + m * 2.0 ** -40 + 2.0 ** -140


@pytest.mark.parametrize("T,heads,d,rot,layout,scaling,dtype,theta", [
    (1, 1, 2, 2, "half", None, torch.float32, 10.0),
    (5, 3, 128, 128, "half", None, torch.bfloat16, 5e5),
    (37, 2, 128, 64, "interleaved", PARTS, torch.bfloat16, 5e5),
    (7, 5, 96, 48, "half", YARN, torch.float32, 1e4),
    (9, 4, 64, 32, "half", dict(kind="linear", factor=3.0), torch.bfloat16, 1e6),
    (6, 2, 256, 256, "interleaved", YARN, torch.float32, 5e5),
    (3, 2, 30, 22, "half", None, torch.bfloat16, 5e5),            # no vector path: odd sizes
    (3, 2, 72, 10, "interleaved", None, torch.bfloat16, 5e5),     # a vector that straddles the turned part's end
    (700, 1, 64, 64, "half", PARTS, torch.float32, 5e5),          # several tokens per CTA step
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_fp64(c, T, heads, d, rot, layout, scaling, dtype, theta, inverse):
    x = _randn(T, heads, d, seed=T + d, dtype=dtype)
    pos = torch.randint(-1000, 1 << 21, (T,), generator=torch.Generator().manual_seed(T))
    pos[0] = (1 << 40) + 12345                                    # far beyond 32 bits
    plan = c.mxs_rope_plan(rot, theta, layout, scaling)
    for odt in (torch.float32, torch.bfloat16):
        y = c.mxs_rope(x, pos.cuda(), plan, inverse=inverse, dtype=odt)
        # the plan's steps are rounded to 2^-64 turns: 2^40 * 2^-65 turns at the far position
        ref = serving.rope(_np(x), pos.tolist(), rot, theta, layout, scaling, inverse)
        tol = _rope_bound(_np(x), ref, odt == torch.bfloat16)
        tol[0] += 7 * 2.0 ** -22 * np.abs(_np(x)[0]).max()        # 2 pi 2^40 2^-65, and long double's 2^-64 of 2^40 radians
        assert np.all(np.abs(_np(y) - ref) <= tol)


def test_rope_strides_in_place_and_unaligned(c):
    plan, pos = c.mxs_rope_plan(64, layout="half"), torch.arange(50, 59, device="cuda")
    qkv = _randn(9, 6 * 64 + 3, seed=1, dtype=torch.bfloat16)
    x = qkv[:, 3:].unflatten(1, (6, 64))                          # odd pitch, 2-byte aligned rows
    want = c.mxs_rope(x.contiguous(), pos, plan)
    assert torch.equal(c.mxs_rope(x, pos, plan), want)
    head_major = torch.empty(6, 9, 64, dtype=torch.bfloat16, device="cuda")
    c.mxs_rope(x, pos, plan, out=head_major.transpose(0, 1))
    assert torch.equal(head_major.transpose(0, 1), want)
    rest = qkv[:, :3].clone()
    assert c.mxs_rope(x, pos, plan, out=x) is x
    assert torch.equal(x, want) and torch.equal(qkv[:, :3], rest)
    assert c.mxs_rope(x[:0], pos[:0], plan).shape == (0, 6, 64)


def test_rope_inverse_is_the_gradient(c):
    """<rope(x), g> = <x, rope^-1(g)>, and the inverse gives what differences
    of <rope(x), g> do.  fp32 roundings: 2^-24 of each of n products."""
    plan, pos = c.mxs_rope_plan(64, scaling=YARN), torch.tensor([3, 99999], device="cuda")
    x, g = _randn(2, 3, 128, seed=2), _randn(2, 3, 128, seed=3)
    dx = c.mxs_rope(g, pos, plan, inverse=True)
    lhs = (c.mxs_rope(x, pos, plan).double() * g.double()).sum()
    rhs = (x.double() * dx.double()).sum()
    n = (x.double().abs() * dx.double().abs()).sum() * 3
    assert abs(lhs - rhs) <= 2.0 ** -24 * 2 * n
    for i in (0, 17, 40, 63, 64, 127):
        e = torch.zeros_like(x)
        e[1, 2, i] = 1.0
        # linear: the difference of step one, f(x + e) - f(x) with f(e) alone
        diff = (c.mxs_rope(e, pos, plan).double() * g.double()).sum()
        assert abs(diff - dx[1, 2, i].double()) <= 2.0 ** -23 * 2 * g[1, 2].double().abs().max() * 2


# ------------------------------------------------------------------- cache
def _codes(cache):
    g = 2 if cache.K.layout.c.seg[2].k_real else 0
    return [(t.code_rows(g), t.scale_rows(g)) for t in (cache.K, cache.V)]


def _quantized(x, bits):
    """The oracle's codes and scales of fp32 rows."""
    d = x.shape[-1]
    counts = (0, 0, d) if bits == 4 else (d, 0, 0)
    cs, ss = oracle.quantize_rows(np.asarray(x, dtype=np.float64).reshape(-1, d), None, counts)
    return cs[2 if bits == 4 else 0], ss[2 if bits == 4 else 0]


@pytest.mark.parametrize("T,n_kvh,d,bits,rot,layout,dtype", [
    (1, 1, 32, 4, 0, "half", torch.bfloat16),
    (5, 8, 128, 4, 128, "half", torch.bfloat16),
    (601, 2, 128, 4, 64, "half", torch.float32),         # several tokens per step; a turned and a copied run
    (13, 3, 64, 8, 32, "interleaved", torch.float32),
    (13, 3, 64, 8, 32, "half", torch.bfloat16),          # pairs inside a block
    (7, 2, 96, 4, 96, "half", torch.float32),            # pairs across blocks of 32
    (4, 2, 256, 8, 192, "half", torch.bfloat16),
    (4, 1, 192, 4, 20, "interleaved", torch.bfloat16),
    (1003, 5, 64, 8, 32, "interleaved", torch.float32),  # tokens that lie across the warps of a CTA
    (1207, 3, 128, 4, 128, "half", torch.bfloat16),
    (2501, 8, 128, 8, 128, "half", torch.bfloat16),
])
def test_write_matches_oracle_and_read_returns_it(c, T, n_kvh, d, bits, rot, layout, dtype):
    n_slots = 2 * T + 3
    cache = c.kv_cache_empty(n_slots, n_kvh, d, bits)
    k, v = _randn(T, n_kvh, d, seed=d + T, dtype=dtype), _randn(T, n_kvh, d, seed=d + T + 1, dtype=dtype)
    k[:, :, ::17] *= 30.0
    v[T // 2] = 0.0                                               # zero blocks
    v[0, 0, :32] = 1e-39 if dtype == torch.float32 else 2.0 ** -130   # a subnormal block
    slot = torch.randperm(n_slots, generator=torch.Generator().manual_seed(T))[:T].cuda()
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(1)).cuda()
    plan = c.mxs_rope_plan(rot, layout=layout, scaling=YARN) if rot else None
    for t in (cache.K, cache.V):
        for b in (*t.codes, *t.scales):
            if b is not None:
                b.fill_(0xA5)
    before = [(x.clone(), y.clone()) for x, y in _codes(cache)]
    c.mxs_kv_write(k, v, cache, slot, pos=pos if rot else None, rope=plan)
    c.mxs_sync()
    kr = c.mxs_rope(k, pos, plan, dtype=torch.float32) if rot else k.float()
    if rot:
        # mxs_rope to fp32 is what the 64-bit rotation rounds to
        ref = serving.rope(_np(k), pos.tolist(), rot, 5e5, layout, YARN).astype(np.float32)
        assert np.mean(_np(kr).astype(np.float32) != ref) < 1e-3
    at = (slot[:, None] * n_kvh + torch.arange(n_kvh, device="cuda")).reshape(-1)
    rest = torch.ones(n_slots * n_kvh, dtype=torch.bool, device="cuda")
    rest[at] = False
    for (codes, scales), (c0, s0), x in zip(_codes(cache), before, (kr, v.float())):
        oc, os_ = _quantized(x.cpu().numpy(), bits)
        assert np.array_equal(codes[at].cpu().numpy(), oc) and np.array_equal(scales[at].cpu().numpy(), os_)
        assert torch.equal(codes[rest], c0[rest]) and torch.equal(scales[rest], s0[rest])
    # reading back: what the codes stand for, in any order and more than once
    pick = torch.cat([slot.flip(0), slot[:1], slot.new_tensor([-1])])
    for odt in (torch.float32, torch.bfloat16):
        out = tuple(torch.full((T + 2, n_kvh, d), 7.0, dtype=odt, device="cuda") for _ in range(2))
        c.mxs_kv_read(cache, pick, out=out)
        for o, t in zip(out, (cache.K, cache.V)):
            vals = c.mxs_dequantize(t).view(n_slots, n_kvh, d)
            assert torch.equal(o[:-1].float(), vals[pick[:-1]].to(odt).float()) and torch.all(o[-1] == 7.0)
    c.mxs_sync()


def test_write_is_rope_then_quantize(c):
    """The fused call gives the bits of mxs_rope to fp32 and mxs_quantize_act,
    from strided and unaligned rows as from dense ones."""
    T, n_kvh, d = 300, 4, 128
    qkv = _randn(T, 4 * n_kvh * d + 1, seed=5, dtype=torch.bfloat16)
    plan, pos = c.mxs_rope_plan(d, scaling=PARTS), torch.arange(T, device="cuda") + 70000
    slot = torch.arange(T, device="cuda")
    lay = c.mxs_layout_make(d, (0, 0, d))
    for off in (0, 1):
        k, v = (qkv[:, off + i * n_kvh * d: off + (i + 1) * n_kvh * d].unflatten(1, (n_kvh, d)) for i in (2, 3))
        cache = c.kv_cache_empty(T, n_kvh, d)
        c.mxs_kv_write(k, v, cache, slot, pos=pos, rope=plan)
        for got, x in zip((cache.K, cache.V), (c.mxs_rope(k, pos, plan, dtype=torch.float32), v.float())):
            want = c.mxtensor_empty(T * n_kvh, lay)
            c.mxs_quantize_act(x.reshape(-1, d).contiguous(), want)
            assert torch.equal(got.code_rows(2), want.code_rows(2))
            assert torch.equal(got.scale_rows(2), want.scale_rows(2))


@pytest.mark.parametrize("bits", [4, 8])
def test_read_of_every_code_at_every_scale(c, bits):
    """Values are code * 2^(scale byte - 127 - bits + 2), from the smallest
    subnormals to overflow."""
    n_slots, d = 256, 64 if bits == 4 else 256
    cache = c.kv_cache_empty(n_slots, 1, d, bits)
    seg = 2 if bits == 4 else 0
    rng = np.random.default_rng(bits)
    for t in (cache.K, cache.V):
        codes = np.stack([rng.permutation(256).astype(np.uint8) for _ in range(n_slots)])[:, : d * bits // 8]
        scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], d // 32, axis=1)
        t.code_rows(seg).copy_(torch.from_numpy(codes).cuda())
        t.scale_rows(seg).copy_(torch.from_numpy(scales).cuda())
    out32 = c.mxs_kv_read(cache, torch.arange(n_slots, device="cuda"), dtype=torch.float32)
    out16 = c.mxs_kv_read(cache, torch.arange(n_slots, device="cuda"))
    for t, a, b in zip((cache.K, cache.V), out32, out16):
        raw = t.code_rows(seg).cpu().numpy()
        q = raw.view(np.int8).astype(np.float64) if bits == 8 else np.stack(
            [((raw & 15) ^ 8).astype(np.float64) - 8, ((raw >> 4) ^ 8).astype(np.float64) - 8], axis=-1).reshape(n_slots, d)
        with np.errstate(over="ignore"):
            want = (q * 2.0 ** (np.arange(256)[:, None] - 127.0 - bits + 2)).astype(np.float32)
        assert np.array_equal(a[:, 0].cpu().numpy(), want)
        assert torch.equal(b[:, 0].cpu(), torch.from_numpy(want).bfloat16())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_write_of_every_scale_and_every_tie(c, bits, dtype):
    """Blocks whose maximum has each exponent that bf16 holds, with values at
    the codes, half-way between two codes and beyond the largest code."""
    d, top = 128, 2 ** (bits - 1)
    e = np.arange(-126, 128)
    steps = np.concatenate([np.arange(0, 2 * top) / 2.0, [top - 0.25]]) / (top / 2)     # in units of 2^e
    steps = steps[:: max(1, len(steps) // 60)]
    pat = np.resize(np.concatenate([steps, -steps]), d)
    pat[::32] = 1.0                                                # the block's exponent is e or above
    x = torch.from_numpy((pat * 2.0 ** e[:, None].astype(np.float64)).astype(np.float32)).cuda().to(dtype)[:, None, :]
    x = torch.cat([x, torch.zeros_like(x[:1])])
    cache = c.kv_cache_empty(x.shape[0], 1, d, bits)
    c.mxs_kv_write(x, -x, cache, torch.arange(x.shape[0], device="cuda"))
    c.mxs_sync()
    for (codes, scales), y in zip(_codes(cache), (x, -x)):
        oc, os_ = _quantized(y.float().cpu().numpy(), bits)
        assert np.array_equal(scales.cpu().numpy(), os_) and np.array_equal(codes.cpu().numpy(), oc)


def test_slots_out_of_range_are_skipped_and_recorded(c):
    cache = c.kv_cache_empty(6, 2, 64)
    k = _randn(4, 2, 64, seed=6, dtype=torch.bfloat16)
    c.mxs_kv_write(k, k, cache, torch.tensor([2, -1, -(1 << 40), 0], device="cuda"))
    c.mxs_sync()                                                  # negative slots are no error
    kk, _ = c.mxs_kv_read(cache, torch.arange(6, device="cuda"))
    assert torch.count_nonzero(kk[[1, 3, 4, 5]]) == 0 and torch.count_nonzero(kk[[0, 2]]) > 0
    n0 = [x.clone() for pair in _codes(cache) for x in pair]
    for bad in (6, 1 << 40):
        c.mxs_kv_write(k[:1], k[:1], cache, torch.tensor([bad], device="cuda"))
        with pytest.raises(c.MxsError) as e:
            c.mxs_sync()
        assert e.value.status == 2
        out = (torch.ones(1, 2, 64, device="cuda"), torch.ones(1, 2, 64, device="cuda"))
        c.mxs_kv_read(cache, torch.tensor([bad], device="cuda"), out=out)
        with pytest.raises(c.MxsError):
            c.mxs_sync()
        assert torch.all(out[0] == 1) and torch.all(out[1] == 1)
    assert all(torch.equal(a, b) for a, b in zip(n0, [x for pair in _codes(cache) for x in pair]))
    c.mxs_sync()


# --------------------------------------------------------------- attention
def _trees(counts, words, seed):
    """Masks (rows, words) uint32 of random trees: a token sees its ancestors
    and itself."""
    rng = np.random.default_rng(seed)
    out = []
    for n in counts:
        m = np.zeros((n, words), dtype=np.uint32)
        for i in range(n):
            parent = int(rng.integers(-1, i)) if i else -1
            if parent >= 0:
                m[i] = m[parent]
            m[i, i // 32] |= np.uint32(1 << (i % 32))
        out.append(m)
    return np.concatenate(out) if out else np.zeros((0, words), np.uint32)


def _random_cache(c, n_slots, n_kvh, d, bits, seed):
    cache = c.kv_cache_empty(n_slots, n_kvh, d, bits)
    k, v = (_randn(n_slots, n_kvh, d, seed=seed + i, dtype=torch.bfloat16) for i in range(2))
    c.mxs_kv_write(k, v, cache, torch.arange(n_slots, device="cuda"))
    return cache


def _decoded(c, cache):
    return [_np(x) for x in c.mxs_kv_read(cache, torch.arange(cache.n_slots, device="cuda"), dtype=torch.float32)]


def _check(c, got, lse, q, cache, qs, ln, pages, page, sm, mask, bf16):
    K, V = _decoded(c, cache)
    ref, rl, spread = serving.attn_tree(_np(q), K, V, qs, ln, pages, page, sm, mask)
    got, lse = _np(got), _np(lse)
    d, n = q.shape[2], max([int(x) for x in ln] + [0]) + q.shape[0]
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    empty = np.isneginf(rl)
    assert np.all(got[empty] == 0)
    s = spread * sm
    ds = (d * 2.0 ** -24 + 3 * 2.0 ** -23) * s
    rel = 2 * (ds + 2.0 ** -22 + n * 2.0 ** -24) + (2.0 ** -8 if bf16 else 2.0 ** -16)
    tol = rel[..., None] * np.abs(V).max() + np.abs(ref) * (2.0 ** -8 if bf16 else 2.0 ** -24)
    err = np.abs(got - ref)
    assert np.all(err <= tol), (np.nanmax(err / tol), np.unravel_index(np.nanargmax(err / tol), err.shape))
    ok = ~empty
    assert np.all(np.abs(lse - rl)[ok] <= (ds + 2.0 ** -22 + n * 2.0 ** -24 + 2.0 ** -23 * np.abs(rl))[ok])


def _case(c, ctx, counts, n_qh, n_kvh, d, bits, page, causal, seed, q_scale=1.0, spare=0, empty_rows=False):
    """A ragged batch over randomly placed pages."""
    B, max_len = len(ctx), max(a + b for a, b in zip(ctx, counts))
    per = max(1, -(-max_len // page))
    n_slots = (B * per + 2) * page + 3
    rng = np.random.default_rng(seed)
    pages = rng.permutation(B * per + 2)[: B * per].reshape(B, per).astype(np.int32)
    qs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(qs[-1]) + spare
    cache = _random_cache(c, n_slots, n_kvh, d, bits, seed)
    q = (_randn(rows, n_qh, d, seed=seed + 9) * q_scale).to(torch.bfloat16)
    mask = None
    if not causal:
        words = max(1, -(-max(counts) // 32))
        mask = np.concatenate([_trees(counts, words, seed), np.zeros((spare, words), np.uint32)])
        if empty_rows:
            mask[::2] = 0
    tm = None if mask is None else torch.from_numpy(mask.view(np.int32)).cuda()
    batch = c.tree_batch(torch.from_numpy(qs).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                         torch.from_numpy(pages).cuda(), page, max_q=max(counts), max_len=max_len, mask=tm)
    return q, cache, batch, (qs, ctx, pages, page), mask


SHAPES = [
    # ctx, counts, n_qh, n_kvh, d, bits, page, causal
    ([0], [1], 1, 1, 64, 4, 1, True),                             # one token that sees itself
    ([127, 128, 0], [1, 1, 1], 8, 2, 128, 4, 16, True),           # single tokens about a tile's border
    ([40, 0, 300], [5, 7, 1], 8, 2, 128, 4, 16, False),           # trees, one of them without a context
    ([1000, 511], [16, 3], 8, 8, 64, 8, 33, False),               # pages that end inside a tile; one head each
    ([129], [33], 12, 4, 128, 8, 5, False),                       # masks of two words
    ([70, 0, 5], [64, 0, 2], 4, 1, 64, 4, 128, True),             # a chunk; a sequence without drafted tokens
    ([20], [150], 6, 2, 128, 4, 64, True),                        # more rows than a tile takes
    ([300], [9], 32, 2, 128, 4, 7, False),                        # sixteen query heads per K/V head
    ([2100, 1, 900], [2, 2, 2], 10, 5, 64, 4, 512, False),        # several splits for some
    ([95], [70], 7, 1, 64, 8, 1, False),                          # masks of three words, page of one token
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("bf16", [True, False])
def test_attention_matches_fp64(c, shape, bf16):
    *shape, causal = shape
    q, cache, batch, where, mask = _case(c, *shape, causal, seed=sum(shape[0]) + shape[4])
    sm = shape[4] ** -0.5
    out, lse = c.mxs_attn_tree(q, cache, batch, sm, dtype=torch.bfloat16 if bf16 else torch.float32, return_lse=True)
    c.mxs_sync()
    _check(c, out, lse, q, cache, *where, sm, mask, bf16)


@pytest.mark.parametrize("q_scale,sm", [(8.0, 0.3), (40.0, 1.0), (1.0, 0.0), (1.0, -0.2)])
def test_attention_of_sharp_flat_and_negative_scales(c, q_scale, sm):
    q, cache, batch, where, mask = _case(c, [700, 64], [6, 20], 8, 2, 128, 4, 16, False, seed=3, q_scale=q_scale)
    out, lse = c.mxs_attn_tree(q, cache, batch, sm, dtype=torch.float32, return_lse=True)
    K, V = _decoded(c, cache)
    _check(c, out, lse, q, cache, *where, sm, mask, False) if sm >= 0 else _check_negative(c, out, lse, q, cache, where, sm, mask)


def _check_negative(c, out, lse, q, cache, where, sm, mask):
    """A negative scale is that of the negated query."""
    K, V = _decoded(c, cache)
    ref, rl, _ = serving.attn_tree(-_np(q), K, V, *where, -sm, mask)
    assert np.abs(_np(out) - ref).max() <= 1e-3 * np.abs(V).max() and np.abs(_np(lse) - rl).max() <= 1e-3


def test_rising_scores(c):
    """Later tokens score far above all earlier ones: the running maximum is
    overtaken again and again."""
    n_slots, d = 1024, 64
    cache = c.kv_cache_empty(n_slots, 1, d, 8)
    k = torch.zeros(n_slots, 1, d, device="cuda")
    k[:, 0, 0] = torch.arange(n_slots, device="cuda") * 0.25
    c.mxs_kv_write(k, _randn(n_slots, 1, d, seed=8), cache, torch.arange(n_slots, device="cuda"))
    q = torch.zeros(3, 4, d, device="cuda", dtype=torch.bfloat16)
    q[:, :, 0] = torch.tensor([4.0, -4.0, 0.125, 0.0], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (np.array([0, 3]), [1021], [[0]], n_slots, 1.0)
    batch = c.tree_batch(torch.tensor([0, 3], **i32), torch.tensor([1021], **i32), torch.zeros(1, 1, **i32), n_slots,
                         max_q=3, max_len=n_slots)
    for dt in (torch.bfloat16, torch.float32):
        out, lse = c.mxs_attn_tree(q, cache, batch, 1.0, dtype=dt, return_lse=True)
        _check(c, out, lse, q, cache, *args, None, dt == torch.bfloat16)


def test_rows_that_see_nothing_and_rows_of_no_sequence(c):
    q, cache, batch, where, mask = _case(c, [0, 0, 50], [9, 1, 4], 8, 2, 128, 4, 16, False, seed=4, spare=5,
                                         empty_rows=True)
    out = torch.full((q.shape[0], 8, 128), 3.0, device="cuda")
    got, lse = c.mxs_attn_tree(q, cache, batch, 0.1, out=out, return_lse=True)
    assert got is out and torch.all(out[-5:] == 3.0)
    n = q.shape[0] - 5
    _check(c, out[:n], lse[:n], q[:n], cache, *where, 0.1, mask[:n], False)


def test_garbage_in_places_that_no_row_sees(c):
    """Scale bytes of infinities behind the sequences, in masked drafted
    tokens and in other pages leave the result as it was; a NaN query row
    stays alone."""
    q, cache, batch, where, mask = _case(c, [30, 129], [3, 6], 8, 2, 128, 4, 16, False, seed=5)
    qs, ctx, pages, page = where
    mask[3:, 0] &= ~np.uint32(1 << 2)                             # drafted token 2 of sequence 1: seen by none
    batch = c.tree_batch(*[torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (qs, ctx, pages)],
                         page, max_q=6, max_len=135, mask=torch.from_numpy(mask.view(np.int32)).cuda())
    want = c.mxs_attn_tree(q, cache, batch, 0.1)
    used = torch.zeros(cache.n_slots, dtype=torch.bool)
    for b, total in enumerate((33, 135)):
        for p in range(total):
            if not (b == 1 and p == 131):
                used[pages[b][p // page] * page + p % page] = True
    for t in (cache.K, cache.V):
        for buf, byte in ((t.codes[2], 0x77), (t.scales[2], 0xFF)):
            buf.view(cache.n_slots, -1)[~used.cuda()] = byte
    assert torch.equal(c.mxs_attn_tree(q, cache, batch, 0.1), want)
    q2 = q.clone()
    q2[4, 3] = float("nan")
    got = c.mxs_attn_tree(q2, cache, batch, 0.1)
    assert torch.all(torch.isnan(got[4, 3]))
    got[4, 3] = want[4, 3]
    assert torch.equal(got, want)


def test_bad_batches_are_left_out_and_recorded(c):
    q, cache, batch, where, _ = _case(c, [40, 40], [2, 2], 4, 2, 64, 4, 16, True, seed=6)
    want = c.mxs_attn_tree(q, cache, batch, 0.1)
    length, q_start, pages, _ = batch.tensors

    def run(expect):
        out = torch.full_like(want, 5.0)
        c.mxs_attn_tree(q, cache, batch, 0.1, out=out)
        if expect:
            with pytest.raises(c.MxsError) as e:
                c.mxs_sync()
            assert e.value.status == 2
        c.mxs_sync()
        return out
    assert torch.equal(run(False), want)
    for bad in (-1, 41, 1 << 30):                                 # a length below zero or above max_len - n
        length[1] = bad
        out = run(True)
        assert torch.equal(out[:2], want[:2]) and torch.all(out[2:] == 5.0)
    length[1] = 40
    for last in (5, 1 << 30, -4):                                 # more rows than max_q or than q has, or fewer than none
        q_start[2] = last
        out = run(True)
        assert torch.equal(out[:2], want[:2]) and torch.all(out[2:] == 5.0)
    q_start[2] = 4
    for bad in (-1, 1 << 20, (1 << 31) - 1):                      # a page outside the pool: keys and values of zero
        keep = pages[1, 0].item()
        pages[1, 0] = bad
        out = run(True)
        assert torch.equal(out[:2], want[:2]) and torch.all(torch.isfinite(out))
        pages[1, 0] = keep
    assert torch.equal(run(False), want)


def test_strides_streams_and_repeats(c):
    q, cache, batch, _, _ = _case(c, [500, 260], [8, 8], 8, 2, 128, 4, 16, False, seed=7)
    want, wl = c.mxs_attn_tree(q, cache, batch, 0.1, return_lse=True)
    for _ in range(3):
        got, gl = c.mxs_attn_tree(q, cache, batch, 0.1, return_lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    # q out of a fused projection, out head-major
    fused = torch.zeros(16, 12, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = q
    hm = torch.empty(8, 16, 128, dtype=torch.bfloat16, device="cuda")
    c.mxs_attn_tree(fused[:, 2:10], cache, batch, 0.1, out=hm.transpose(0, 1))
    assert torch.equal(hm.transpose(0, 1), want)
    # another stream, memory made by the call, and work queued behind it on the first
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [c.mxs_attn_tree(q, cache, batch, 0.1, stream=side) for _ in range(4)]
    [torch.empty(1 << 20, device="cuda").fill_(1.0) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with torch.cuda.stream(side):
        a = c.mxs_attn_tree(q, cache, batch, 0.1)
    b = c.mxs_attn_tree(q, cache, batch, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,counts", [(torch.bfloat16, [40, 33]), (torch.bfloat16, [9, 2]), (torch.float32, [9, 2])])
def test_outputs_in_unaligned_rows(c, d, dtype, counts):
    """Whole and joined items alike, into rows that allow no wide stores: the
    bits of dense rows, and nothing between them."""
    q, cache, batch, _, _ = _case(c, [1900, 700], counts, 10, 2, d, 4, 16, False, seed=d)
    want = c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dtype)
    room = torch.full((q.shape[0], 10, d + 3), 7.0, dtype=dtype, device="cuda")
    c.mxs_attn_tree(q, cache, batch, 0.1, out=room[:, :, 1: d + 1])
    assert torch.equal(room[:, :, 1: d + 1], want)
    assert torch.all(room[:, :, 0] == 7.0) and torch.all(room[:, :, d + 1:] == 7.0)


MORE = [
    # ctx, counts, n_qh, n_kvh, d, bits, page, causal
    ([2500, 40], [17, 3], 16, 2, 128, 4, 16, False),              # 136 rows: half of the wide form's second half
    ([1500], [40], 32, 4, 64, 8, 33, True),                       # 320 rows: a second row tile with one half
    ([4100], [5], 12, 4, 128, 8, 64, False),                      # 16 columns over 33 tiles
    ([3000, 2900, 10], [9, 10, 1], 6, 2, 64, 4, 7, True),         # 32 columns, parts of items at both ends of a CTA
    ([2600], [20], 6, 2, 128, 8, 128, False),                     # 64 rows of 8 bits
]


@pytest.mark.parametrize("shape", MORE, ids=[str(i) for i in range(len(MORE))])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("sm", [0.11, -0.07])
def test_long_items_and_both_signs_of_the_scale(c, shape, bf16, sm):
    *shape, causal = shape
    q, cache, batch, (qs, ctx, pages, page), mask = _case(c, *shape, causal, seed=sum(shape[0]) + shape[4])
    out, lse = c.mxs_attn_tree(q, cache, batch, sm, dtype=torch.bfloat16 if bf16 else torch.float32, return_lse=True)
    c.mxs_sync()
    # a negative scale is that of the negated query
    _check(c, out, lse, q if sm > 0 else -q, cache, qs, ctx, pages, page, abs(sm), mask, bf16)


@pytest.mark.parametrize("n_qh", [2, 12, 40])                    # 16 and 64 columns, the wide form
def test_scores_that_rise_over_many_tiles(c, n_qh):
    """The reference of the weights moves again and again, and output periods
    end between."""
    n_slots, d, n = 4096, 64, 5
    cache = c.kv_cache_empty(n_slots, 1, d, 8)
    k = torch.zeros(n_slots, 1, d, device="cuda")
    k[:, 0, 0] = torch.arange(n_slots, device="cuda") * 0.25
    c.mxs_kv_write(k, _randn(n_slots, 1, d, seed=18), cache, torch.arange(n_slots, device="cuda"))
    q = torch.zeros(n, n_qh, d, device="cuda", dtype=torch.bfloat16)
    q[:, :, 0] = (torch.arange(n * n_qh, device="cuda").view(n, n_qh) % 7 - 3.0) * 0.5
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = c.tree_batch(torch.tensor([0, n], **i32), torch.tensor([n_slots - n], **i32), torch.zeros(1, 1, **i32), n_slots,
                         max_q=n, max_len=n_slots)
    for dt in (torch.bfloat16, torch.float32):
        out, lse = c.mxs_attn_tree(q, cache, batch, 1.0, dtype=dt, return_lse=True)
        _check(c, out, lse, q, cache, np.array([0, n]), [n_slots - n], [[0]], n_slots, 1.0, None, dt == torch.bfloat16)


def test_many_small_sequences(c):
    """More items than CTAs, most of them within one tile, empty ones between."""
    rng = np.random.default_rng(90)
    ctx = [int(x) for x in rng.integers(0, 200, 301)]
    counts = [int(x) for x in rng.integers(0, 4, 301)]
    q, cache, batch, where, mask = _case(c, ctx, counts, 4, 2, 64, 4, 16, True, seed=91)
    for dt in (torch.bfloat16, torch.float32):
        out, lse = c.mxs_attn_tree(q, cache, batch, 0.2, dtype=dt, return_lse=True)
        _check(c, out, lse, q, cache, *where, 0.2, None, dt == torch.bfloat16)
    # one call of the whole batch is what calls of its sequences give
    i32 = dict(dtype=torch.int32, device="cuda")
    qs, _, pages, page = where
    for b in (0, 150, 300):
        if counts[b] == 0:
            continue
        one = c.tree_batch(torch.tensor([0, counts[b]], **i32), torch.tensor([ctx[b]], **i32),
                           torch.tensor(pages[b: b + 1], **i32), page, max_q=counts[b], max_len=ctx[b] + counts[b])
        alone = c.mxs_attn_tree(q[qs[b]: qs[b + 1]], cache, one, 0.2, dtype=torch.float32)
        assert (alone - out[qs[b]: qs[b + 1]]).abs().max() <= 1e-5


def test_forms_of_a_call_agree(c):
    """What the extension marshals and what the general path does: given
    outputs, streams and types, outputs that allow no vector stores."""
    for counts, n_qh in (([8, 8], 8), ([40, 3], 32)):             # the second: the wide form
        q, cache, batch, _, _ = _case(c, [500, 260], counts, n_qh, 2, 128, 4, 16, False, seed=17)
        rows = q.shape[0]
        for dt in (torch.bfloat16, torch.float32):
            want, wl = c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dt, return_lse=True)
            odd = torch.full((rows, n_qh * 128 + 3), 7.0, dtype=dt, device="cuda")
            out = odd[:, 1: 1 + n_qh * 128].unflatten(1, (n_qh, 128))
            got, gl = c.mxs_attn_tree(q, cache, batch, 0.1, out=out, return_lse=True)
            assert torch.equal(got, want) and torch.equal(gl, wl)
            assert torch.all(odd[:, 0] == 7.0) and torch.all(odd[:, -2:] == 7.0)
            got = c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dt, stream=torch.cuda.current_stream())
            assert torch.equal(got, want)
    x, pos, plan = _randn(5, 3, 128, seed=1), torch.arange(5, device="cuda"), c.mxs_rope_plan(128)
    for dt in (None, torch.bfloat16):
        want = c.mxs_rope(x, pos, plan, dtype=dt)
        assert torch.equal(c.mxs_rope(x, pos, plan, out=torch.empty_like(want)), want)
        assert torch.equal(c.mxs_rope(x, pos, plan, dtype=dt, stream=torch.cuda.current_stream()), want)
    small = c.kv_cache_empty(5, 3, 128, 8)
    c.mxs_kv_write(x, x, small, pos, pos=pos, rope=plan)
    first = [t.clone() for t in c.mxs_kv_read(small, pos, dtype=torch.float32)]
    c.mxs_kv_write(x, x, small, pos, pos=pos, rope=plan, stream=torch.cuda.current_stream())
    again = c.mxs_kv_read(small, pos, dtype=torch.float32, stream=torch.cuda.current_stream())
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    with pytest.raises(ValueError):
        c.mxs_rope(x, pos.int(), plan)
    with pytest.raises(ValueError):
        c.mxs_rope(x, pos.cpu(), plan)
    with pytest.raises(TypeError):
        c.mxs_rope(x.half(), pos, plan)
    with pytest.raises(ValueError):
        c.mxs_kv_write(x, x, small, pos[:4])
    with pytest.raises(ValueError):
        c.mxs_kv_read(small, pos[None])
    with pytest.raises(c.MxsError) as e:
        c.mxs_rope(x, pos, c.mxs_rope_plan(256))
    assert e.value.status == 2


def test_a_workspace_of_exactly_the_size(c):
    q, cache, batch, _, _ = _case(c, [5000, 700], [4, 60], 8, 2, 128, 4, 16, True, seed=19)
    for dt in (torch.bfloat16, torch.float32):
        need = c.mxs_attn_tree_workspace_bytes(q, cache, batch, dt)
        assert need > 0
        buf = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        first = -buf.data_ptr() % 256
        want = c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dt)
        assert torch.equal(c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dt, workspace=buf[first: first + need]), want)
        assert torch.all(buf[:first] == 0xA5) and torch.all(buf[first + need:] == 0xA5)
        with pytest.raises(c.MxsError) as e:
            c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dt, workspace=buf[first: first + need - 1])
        assert e.value.status == 9


def test_two_streams_at_once(c):
    """Calls that overlap, each with memory of its own."""
    cases = [_case(c, [1500, 300], [6, 9], 8, 2, 128, 4, 16, False, seed=20),
             _case(c, [900], [70], 16, 2, 64, 8, 16, True, seed=21)]
    want = [c.mxs_attn_tree(q, cache, batch, 0.1) for q, cache, batch, *_ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, (s, (q, cache, batch, *_)) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                outs[i].append(c.mxs_attn_tree(q, cache, batch, 0.1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for os, w in zip(outs, want) for o in os)


def test_workspace_refusals(c):
    q, cache, batch, _, _ = _case(c, [5000], [4], 8, 2, 128, 4, 16, True, seed=8)
    need = c.mxs_attn_tree_workspace_bytes(q, cache, batch)
    if need:
        with pytest.raises(c.MxsError) as e:
            c.mxs_attn_tree(q, cache, batch, 0.1, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == 9
    with pytest.raises(ValueError):
        c.mxs_attn_tree(q[:, :, :64], cache, batch, 0.1)
    with pytest.raises(ValueError):
        c.mxs_attn_tree(q, cache, batch, 0.1, out=torch.empty(4, 4, 128, device="cuda"))


# ---------------------------------------------------------------- together
def _step(c, s):
    """One speculative step: turn the drafted queries, write the drafted keys
    and values, attend."""
    q = c.mxs_rope(s["q"], s["pos"], s["plan"])
    c.mxs_kv_write(s["k"], s["v"], s["cache"], s["slot"], pos=s["pos"], rope=s["plan"])
    return c.mxs_attn_tree(q, s["cache"], s["batch"], s["sm"], workspace=s["ws"])


def _serving_state(c, ctx, counts, seed, n_qh=8, n_kvh=2, d=128, page=16):
    B, total = len(ctx), [a + b for a, b in zip(ctx, counts)]
    per = -(-max(total) // page)
    rng = np.random.default_rng(seed)
    pages = rng.permutation(B * per).reshape(B, per)
    rows = sum(counts)
    words = -(-max(counts) // 32)
    mask = _trees(counts, words, seed)
    # a drafted token's position is its depth in the tree
    depth = np.array([bin(int.from_bytes(m.tobytes(), "little")).count("1") - 1 for m in mask])
    base = np.repeat(ctx, counts)
    place = base + np.concatenate([np.arange(n) for n in counts])
    which = np.repeat(np.arange(B), counts)
    dev = dict(device="cuda")
    s = dict(q=_randn(rows, n_qh, d, seed=seed, dtype=torch.bfloat16), k=_randn(rows, n_kvh, d, seed=seed + 1, dtype=torch.bfloat16),
             v=_randn(rows, n_kvh, d, seed=seed + 2, dtype=torch.bfloat16), pos=torch.tensor(base + depth, **dev),
             slot=torch.tensor(pages[which, place // page] * page + place % page, **dev),
             plan=c.mxs_rope_plan(d, scaling=PARTS), sm=d ** -0.5)
    s["cache"] = c.kv_cache_empty(B * per * page, n_kvh, d)
    for b in range(B):                                            # the context, as a prompt's write
        p = np.arange(ctx[b])
        sl = torch.tensor(pages[b][p // page] * page + p % page, **dev)
        c.mxs_kv_write(_randn(ctx[b], n_kvh, d, seed=seed + 10 + b, dtype=torch.bfloat16),
                       _randn(ctx[b], n_kvh, d, seed=seed + 20 + b, dtype=torch.bfloat16), s["cache"], sl,
                       pos=torch.arange(ctx[b], **dev), rope=s["plan"])
    qs = np.concatenate([[0], np.cumsum(counts)])
    i32 = dict(dtype=torch.int32, device="cuda")
    s["batch"] = c.tree_batch(torch.tensor(qs, **i32), torch.tensor(ctx, **i32), torch.tensor(pages, **i32), page,
                              max_q=max(counts), max_len=max(total), mask=torch.from_numpy(mask.view(np.int32)).cuda())
    s["ws"] = c.attn_tree_workspace(s["q"], s["cache"], s["batch"])
    s["where"] = (qs, ctx, pages, page)
    s["mask"] = mask
    return s


def test_a_speculative_step(c):
    s = _serving_state(c, [333, 90], [12, 7], seed=30)
    out = _step(c, s)
    c.mxs_sync()
    qr = c.mxs_rope(s["q"], s["pos"], s["plan"])
    lse = c.mxs_attn_tree(qr, s["cache"], s["batch"], s["sm"], return_lse=True)[1]
    _check(c, out, lse, qr, s["cache"], *s["where"], s["sm"], s["mask"], True)


def test_a_step_captured_and_replayed_with_new_contents(c):
    """Two captured steps with a workspace each, replayed after their inputs
    changed, against eager calls on the same contents."""
    states = [_serving_state(c, [333, 90], [12, 7], seed=31), _serving_state(c, [700], [30], seed=41)]
    graphs = []
    for s in states:
        _step(c, s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s["out"] = _step(c, s)
        graphs.append(g)
    for trial in range(2):
        for s in states:
            s["q"].copy_(_randn(*s["q"].shape, seed=50 + trial))
            s["k"].copy_(_randn(*s["k"].shape, seed=60 + trial))
            s["pos"].add_(1)
            s["batch"].tensors[0].sub_(1)                         # a shorter context
        want = []
        for s in states:
            want.append(_step(c, s).clone())
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s["out"], w) for s, w in zip(states, want))
    c.mxs_sync()


def test_decode_attention_agrees_on_a_contiguous_cache(c):
    """The cache that mxs_kv_write fills is the one mxs_attn_decode reads:
    both calls give the same step."""
    T, n_qh, n_kvh, d = 1500, 8, 2, 128
    cache = _random_cache(c, T, n_kvh, d, 4, seed=70)
    q = _randn(1, n_qh, d, seed=72, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = c.tree_batch(torch.tensor([0, 1], **i32), torch.tensor([T - 1], **i32), torch.zeros(1, 1, **i32), T,
                         max_q=1, max_len=T)
    a = c.mxs_attn_tree(q, cache, batch, d ** -0.5, dtype=torch.float32)[0]
    b = c.mxs_attn_decode(q[0], cache.K, cache.V, T, n_kvh, d ** -0.5)
    vmax = c.mxs_dequantize(cache.V).abs().max()
    # each is within 5e-4 of max|V| of the exact step (2^-16 weights, fp32 sums over 1500 tokens)
    assert (a - b).abs().max() <= 2 * 5e-4 * vmax


def test_slots_beyond_four_gigabytes(c):
    """A pool whose code bytes pass 2^32: rows at its far end."""
    n_kvh, d = 8, 128
    n_slots = (1 << 32) // (n_kvh * 64) + 5000
    cache = c.kv_cache_empty(n_slots, n_kvh, d)
    T, page = 40, 8
    slot = torch.arange(n_slots - 96, n_slots - 96 + T, device="cuda")
    k, v = (_randn(T, n_kvh, d, seed=80 + i, dtype=torch.bfloat16) for i in range(2))
    c.mxs_kv_write(k, v, cache, slot)
    small = c.kv_cache_empty(T, n_kvh, d)
    c.mxs_kv_write(k, v, small, torch.arange(T, device="cuda"))
    far, near = c.mxs_kv_read(cache, slot), c.mxs_kv_read(small, torch.arange(T, device="cuda"))
    assert all(torch.equal(a, b) and torch.count_nonzero(a) > 0 for a, b in zip(far, near))
    assert n_slots % page == 0
    i32 = dict(dtype=torch.int32, device="cuda")
    q = _randn(3, 8, d, seed=83, dtype=torch.bfloat16)
    outs = []
    for cc, first in ((cache, (n_slots - 96) // page), (small, 0)):
        pages = (first + torch.arange(T // page, device="cuda")).to(torch.int32)[None]
        batch = c.tree_batch(torch.tensor([0, 3], **i32), torch.tensor([T - 3], **i32), pages, page, max_q=3, max_len=T)
        outs.append(c.mxs_attn_tree(q, cc, batch, 0.1))
    c.mxs_sync()
    assert torch.equal(*outs)
