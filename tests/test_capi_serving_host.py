"""Host checks of the serving calls: plans, and refusals before any launch.
The refusals pass made-up device addresses and run only where no CUDA device
exists."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import serving

fake_pointers = pytest.mark.skipif(torch.cuda.is_available(),
                                   reason="passes made-up device addresses: CPU hosts only")
X, O, POS, SLOT, WS = 1 << 24, 1 << 28, 1 << 21, 1 << 22, 1 << 30


@pytest.fixture(scope="module")
def c():
    from mx_microscaling_mixed_b200 import build
    build.build()
    from mx_microscaling_mixed_b200 import capi
    return capi


SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="parts", factor=8.0, low=1.0, high=4.0, orig_len=8192),
            dict(kind="yarn", factor=16.0, orig_len=4096), dict(kind="yarn", factor=1.0, orig_len=100, beta_slow=2.0)]


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("rot,theta", [(2, 10.0), (64, 1e4), (128, 5e5), (256, 1e6)])
def test_plan_steps(c, rot, theta, scaling):
    p = c.mxs_rope_plan(rot, theta, "interleaved", scaling).c
    f, gain = serving.rope_frequencies(rot, theta, scaling)
    assert (p.rot, p.layout) == (rot, 1) and math.isclose(p.gain, gain, rel_tol=1e-15)
    got = np.array([int(s) for s in p.step[: rot // 2]], dtype=np.longdouble) / np.longdouble(2) ** 64
    # the steps are rounded to 2^-64; long double carries the rest to about 2^-62 relative
    want = f / (np.longdouble(2) * np.longdouble("3.14159265358979323846264338327950288"))
    assert np.all(np.abs(got - want) <= 2.0 ** -64 + want * 2.0 ** -60)
    assert all(s == 0 for s in p.step[rot // 2:])


def test_plan_refusals(c):
    for bad in (dict(rot=3), dict(rot=0), dict(rot=258), dict(theta=1.0), dict(theta=float("nan")),
                dict(theta=float("inf")), dict(scaling=dict(kind="linear", factor=0.5)),
                dict(scaling=dict(kind="linear", factor=float("nan"))),
                dict(scaling=dict(kind="parts", factor=8.0, low=4.0, high=4.0, orig_len=8192)),
                dict(scaling=dict(kind="parts", factor=8.0, low=0.0, high=4.0, orig_len=8192)),
                dict(scaling=dict(kind="yarn", factor=8.0, orig_len=0))):
        with pytest.raises(c.MxsError) as e:
            c.mxs_rope_plan(**{"rot": 64, **bad})
        assert e.value.status == 1
    for bad in (dict(layout="other"), dict(scaling=dict(kind="other", factor=2.0)),
                dict(scaling=dict(kind="linear", factor=2.0, low=1.0)), dict(scaling=dict(kind="parts", factor=2.0))):
        with pytest.raises(ValueError):
            c.mxs_rope_plan(64, **bad)
    with pytest.raises(ValueError):
        c.kv_cache_empty(4, 1, 64, bits=6, device="cpu")


def _rope(c, plan, xt=1, T=4, heads=2, d=128, ldxt=256, ldxh=128, ldot=256, ldoh=128, x=X, pos=POS, out=O, ot=1):
    return c._lib.mxs_rope(x, xt, T, heads, d, ldxt, ldxh, pos, None if plan is None else plan.ptr, 0, out, ot, ldot,
                           ldoh, None)


@fake_pointers
def test_rope_refusals(c):
    p = c.mxs_rope_plan(128)
    assert _rope(c, None) == 1 and _rope(c, p, T=-1) == 1 and _rope(c, p, x=None) == 1 and _rope(c, p, pos=None) == 1
    assert _rope(c, p, xt=3) == 4 and _rope(c, p, ot=-1) == 4
    assert _rope(c, p, d=64, ldxh=64) == 2                       # rot > d
    assert _rope(c, p, d=129) == 2 and _rope(c, p, d=258) == 2
    assert _rope(c, p, ldot=128) == 2 and _rope(c, p, ldoh=127) == 2 and _rope(c, p, ldoh=0) == 2
    assert _rope(c, p, ldxt=-1) == 2
    assert _rope(c, p, out=X, ot=0) == 2 and _rope(c, p, out=X, ldot=512) == 2    # in place: same type and strides
    assert _rope(c, p, T=0, x=None, out=None) == 0 and _rope(c, p, heads=0) == 0
    bad = c.mxs_rope_plan(128)
    bad.c.rot = 300
    assert _rope(c, bad) == 1


def _cache(c, rows=64, n_kvh=2, d=128, bits=4, rows_v=None, bits_v=None):
    def one(rows, bits, base):
        lay = c.mxs_layout_make(d, (0, 0, d) if bits == 4 else (d, 0, 0) if bits == 8 else (0, d, 0))
        t = c.MXTensorC()
        t.rows, t.lay = rows, lay.c
        cp, _, sp, _ = c.mxs_mxtensor_bytes(rows, lay)
        for g in range(3):
            t.code_pitch[g], t.scale_pitch[g] = cp[g], sp[g]
            if cp[g]:
                t.codes[g], t.scales[g] = base, base + (1 << 20)
        return t
    return c.KVCacheC(one(rows, bits, 1 << 32), one(rows_v or rows, bits_v or bits, 1 << 33), n_kvh)


def _write(c, cache, dt=1, T=4, k=X, v=O, slot=SLOT, pos=None, plan=None, ld=128):
    return c._lib.mxs_kv_write(k, 2 * ld, ld, v, 2 * ld, ld, dt, T, slot, pos, None if plan is None else plan.ptr,
                               ctypes.addressof(cache), None)


def _read(c, cache, ot=1, T=4, k=X, v=O, slot=SLOT, ldt=256, ldh=128):
    return c._lib.mxs_kv_read(ctypes.addressof(cache), T, slot, k, ldt, ldh, v, ldt, ldh, ot, None)


@fake_pointers
def test_cache_refusals(c):
    good, plan = _cache(c), c.mxs_rope_plan(128)
    for call in (_write, _read):
        assert call(c, _cache(c, n_kvh=0)) == 1
        assert call(c, _cache(c, rows=63)) == 2                  # not whole slots
        assert call(c, _cache(c, rows_v=62)) == 2 and call(c, _cache(c, bits_v=8)) == 2
        assert call(c, _cache(c, bits=6)) == 2                   # 6-bit caches are not served
        assert call(c, _cache(c, d=48)) == 2 and call(c, _cache(c, d=288)) == 2
        assert call(c, good, T=-1) == 1 and call(c, good, slot=None) == 1
        assert call(c, good, T=0, k=None, v=None, slot=None) == 0
        assert call(c, _cache(c, rows=1 << 31, n_kvh=1)) == 2     # slots and a slot's bytes are 32-bit numbers
        wide = _cache(c)
        wide.K.scale_pitch[2] = 1 << 31
        assert call(c, wide) == 2
        mis = _cache(c)
        mis.V.codes[2] += 8
        assert call(c, mis) == 3
    assert _write(c, good, dt=2) == 4 and _read(c, good, ot=2) == 4
    assert _write(c, good, k=None) == 1 and _write(c, good, plan=plan) == 1      # rope without positions
    assert _write(c, _cache(c, d=64), plan=plan, pos=POS) == 2                   # rot > d
    assert _read(c, good, k=None, v=None) == 1
    assert _read(c, good, ldh=0) == 2 and _read(c, good, ldt=64) == 2 and _read(c, good, ldt=128) == 2


def _tree(c, cache, q=X, n_qh=8, ldqt=1024, ldqh=128, out=O, ot=1, ldot=1024, ldoh=128, scale=0.1, ws=WS, ws_bytes=1 << 40,
          **kw):
    f = dict(B=2, rows=6, max_q=3, max_len=40, q_start=POS, length=SLOT, pages=SLOT + 4096, ldp=10, page_size=4,
             mask=SLOT + 8192, ldm=1)
    f.update(kw)
    b = c.TreeBatchC(*[f[n] for n, _ in c.TreeBatchC._fields_])
    return c._lib.mxs_attn_tree(q, n_qh, ldqt, ldqh, ctypes.addressof(cache), ctypes.addressof(b), scale, out, ot, ldot,
                                ldoh, None, ws, ws_bytes, None)


@fake_pointers
def test_tree_refusals(c):
    good = _cache(c)
    assert _tree(c, _cache(c, d=96), ldqh=96) == 2               # heads of 64 or 128
    assert _tree(c, good, n_qh=7) == 2 and _tree(c, good, n_qh=0) == 1 and _tree(c, good, n_qh=65536) == 2
    assert _tree(c, good, B=-1) == 1 and _tree(c, good, rows=-1) == 1 and _tree(c, good, B=65536) == 2
    assert _tree(c, good, max_q=41) == 2                         # more drafted tokens than tokens
    assert _tree(c, good, max_len=41) == 2                       # more tokens than ldp pages hold
    assert _tree(c, good, page_size=0) == 2 and _tree(c, good, ldp=-1) == 2
    assert _tree(c, good, max_q=33, ldm=1) == 2                  # mask rows too short
    assert _tree(c, good, ot=7) == 4 and _tree(c, good, scale=float("inf")) == 1
    assert _tree(c, good, q=X + 2) == 3 and _tree(c, good, ldqt=1028) == 3 and _tree(c, good, ldqh=132) == 3
    assert _tree(c, good, ldot=512) == 2 and _tree(c, good, ldoh=64) == 2
    for name in ("q_start", "length", "pages"):
        assert _tree(c, good, **{name: None}) == 1
    assert _tree(c, good, q=None) == 1 and _tree(c, good, out=None) == 1
    assert _tree(c, good, max_q=0, q=None) == 0 and _tree(c, good, B=0) == 0 and _tree(c, good, rows=0) == 0


def test_tree_batch_refusals(c):
    i32 = torch.int32
    qs, ln, pg = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 5, dtype=i32)
    c.tree_batch(qs, ln, pg, 16, max_q=4, max_len=80)
    for args, kw in (((qs[:2], ln, pg, 16), {}), ((qs.long(), ln, pg, 16), {}), ((qs, ln, pg[:1], 16), {}),
                     ((qs, ln, pg.t(), 16), {}), ((qs, ln, pg, 16), dict(mask=torch.zeros(4, 1))),
                     ((qs, ln, torch.zeros(2, 10, dtype=i32)[:, ::2], 16), {})):
        with pytest.raises(ValueError):
            c.tree_batch(*args, max_q=4, max_len=80, **kw)
    for kw in (dict(max_q=4, max_len=81), dict(max_q=33, max_len=80, mask=torch.zeros(4, 1, dtype=i32))):
        with pytest.raises(c.MxsError) as e:
            c.tree_batch(qs, ln, pg, 16, **kw)
        assert e.value.status == 2


def test_binding_refusals(c):
    """Shapes and types that the binding itself refuses, with CPU tensors."""
    p, x = c.mxs_rope_plan(64), torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        c.mxs_rope(x, torch.zeros(4, dtype=torch.int64), p)      # not on a GPU
    with pytest.raises(ValueError):
        c.mxs_rope(x.transpose(1, 2), torch.zeros(4, dtype=torch.int64), p)
    cache = c.kv_cache_empty(4, 2, 64, device="cpu")
    slot = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        c.mxs_kv_write(x, x[:, :1], cache, slot)
    with pytest.raises(TypeError):
        c.mxs_kv_write(x, x.bfloat16(), cache, slot)
    with pytest.raises(ValueError):
        c.mxs_kv_write(x, x, cache, slot, rope=p)
    with pytest.raises(TypeError):
        c.mxs_attn_tree(x, cache, None, 0.1)
