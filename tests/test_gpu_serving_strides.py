"""The serving calls on tensors as views leave them: strides beyond 32 bits,
broadcast heads and tokens, head-major memory, tensors of one head or one
token.  Each gives the bits of dense tensors."""
import pytest
import torch

from tests import parity
from tests.test_gpu_serving import _case, _randn

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 64                                                 # elements from a token to the next


@pytest.fixture(scope="module")
def c():
    parity.need_gpu()
    return parity.capi()


def _far(t, room, at=0):
    """t's values in a view of `room` whose tokens are FAR elements apart."""
    v = room.as_strided(t.shape, (FAR, t.shape[2], 1), at)
    v.copy_(t)
    return v


def test_strides_beyond_32_bits(c):
    T, h, d = 3, 4, 64
    room = torch.empty(2 * FAR + 4 * h * d, dtype=torch.bfloat16, device="cuda")
    x, k, v = (_randn(T, h, d, seed=i, dtype=torch.bfloat16) for i in range(3))
    plan, pos, slot = c.mxs_rope_plan(d), torch.arange(T, device="cuda") + 7, torch.tensor([4, 0, 2], device="cuda")
    want = c.mxs_rope(x, pos, plan)
    far = _far(x, room)
    assert torch.equal(c.mxs_rope(far, pos, plan), want)
    assert c.mxs_rope(far, pos, plan, out=far) is far and torch.equal(far, want)
    near = c.kv_cache_empty(5, h, d)
    c.mxs_kv_write(k, v, near, slot, pos=pos, rope=plan)
    kv = c.mxs_kv_read(near, slot)
    other = c.kv_cache_empty(5, h, d)
    c.mxs_kv_write(_far(k, room), _far(v, room, h * d), other, slot, pos=pos, rope=plan)
    out = (_far(torch.zeros_like(k), room, 2 * h * d), _far(torch.zeros_like(v), room, 3 * h * d))
    c.mxs_kv_read(other, slot, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, kv))
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = c.tree_batch(torch.tensor([0, T], **i32), torch.tensor([2], **i32), torch.zeros(1, 1, **i32), 5, max_q=T, max_len=5)
    for rep in (1, 32):                                              # (the second: the wide form)
        q = _randn(T, h * rep, d, seed=9, dtype=torch.bfloat16)
        big = room if rep == 1 else torch.empty(2 * FAR + 2 * q.shape[1] * d, dtype=torch.bfloat16, device="cuda")
        want = c.mxs_attn_tree(q, near, batch, 0.3)
        got = _far(torch.zeros_like(q), big, q.shape[1] * d)
        c.mxs_attn_tree(_far(q, big), near, batch, 0.3, out=got)
        assert torch.equal(got, want)
    c.mxs_sync()


def test_broadcast_inputs(c):
    T, h, d = 9, 5, 128
    plan, pos, slot = c.mxs_rope_plan(d, layout="interleaved"), torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    for shape in ((T, 1, d), (1, h, d)):
        x = _randn(*shape, seed=1, dtype=torch.bfloat16).expand(T, h, d)
        assert torch.equal(c.mxs_rope(x, pos, plan), c.mxs_rope(x.contiguous(), pos, plan))
        a, b = c.kv_cache_empty(T, h, d), c.kv_cache_empty(T, h, d)
        c.mxs_kv_write(x, x, a, slot, pos=pos, rope=plan)
        c.mxs_kv_write(x.contiguous(), x.contiguous(), b, slot, pos=pos, rope=plan)
        assert all(torch.equal(p, q) for p, q in zip(c.mxs_kv_read(a, slot), c.mxs_kv_read(b, slot)))
        with pytest.raises(c.MxsError) as e:                         # as an output its rows overlap
            c.mxs_rope(x, pos, plan, out=x)
        assert e.value.status == 2
        with pytest.raises(c.MxsError) as e:
            c.mxs_kv_read(a, slot, out=(x, x))
        assert e.value.status == 2
    q, cache, batch, _, _ = _case(c, [300, 20], [8, 5], 8, 2, 128, 4, 16, False, seed=3)
    one = q[:, :1].expand(q.shape)
    assert torch.equal(c.mxs_attn_tree(one, cache, batch, 0.1), c.mxs_attn_tree(one.contiguous(), cache, batch, 0.1))
    with pytest.raises(c.MxsError) as e:
        c.mxs_attn_tree(q, cache, batch, 0.1, out=one)
    assert e.value.status == 2


@pytest.mark.parametrize("T,h", [(1, 6), (7, 1), (1, 1), (7, 6)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_head_major_and_tensors_of_one(c, T, h, dtype):
    d = 64
    plan, pos, slot = c.mxs_rope_plan(32), torch.arange(T, device="cuda") + 100, torch.arange(T, device="cuda").flip(0)
    x = _randn(h, T, d, seed=2, dtype=dtype).transpose(0, 1)
    dense = x.contiguous()
    want = c.mxs_rope(dense, pos, plan)
    assert torch.equal(c.mxs_rope(x, pos, plan), want)
    out = torch.empty(h, T, d, dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(c.mxs_rope(x, pos, plan, out=out), want)
    a, b = c.kv_cache_empty(T, h, d, 8), c.kv_cache_empty(T, h, d, 8)
    c.mxs_kv_write(x, x, a, slot, pos=pos, rope=plan)
    c.mxs_kv_write(dense, dense, b, slot, pos=pos, rope=plan)
    want = c.mxs_kv_read(b, slot, dtype=dtype)
    both = tuple(torch.empty(h, T, d, dtype=dtype, device="cuda").transpose(0, 1) for _ in range(2))
    c.mxs_kv_read(a, slot, out=both)
    assert all(torch.equal(p, q) for p, q in zip(both, want))
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = c.tree_batch(torch.tensor([0, T], **i32), torch.tensor([0], **i32), torch.zeros(1, 1, **i32), T, max_q=T, max_len=T)
    q = x.to(torch.bfloat16)
    assert not (T > 1 and h > 1) or not q.is_contiguous()
    want = c.mxs_attn_tree(q.contiguous(), a, batch, 0.1, dtype=dtype)
    out = torch.empty(h, T, d, dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(c.mxs_attn_tree(q, a, batch, 0.1, out=out), want)
    c.mxs_sync()
