"""Device waits of the attention kernels that run out, without a fault.

With a wait limit far below what a cache tile takes to arrive, the roles of a
CTA give up at whatever wait they are in.  The call returns, mxs_sync reports
MXS_ERR_TIMEOUT once, the products that were issued have finished and the
tensor memory is free again: at the default limit the same call gives the
same bits as before."""
import pytest
import torch

from tests import parity
from tests.test_gpu_serving import _case

pytestmark = pytest.mark.gpu

MXS_ERR_TIMEOUT = 7


@pytest.fixture(scope="module")
def c():
    parity.need_gpu()
    return parity.capi()


FORMS = [
    # ctx, counts, n_qh, n_kvh, d, bits, page, causal, dtype
    ([9000, 7000], [2, 1], 8, 8, 128, 4, 16, True, torch.bfloat16),           # 16 columns, whole and joined items
    ([9000, 7000, 300], [7, 7, 3], 24, 8, 64, 8, 33, False, torch.float32),   # 32 columns, weights in pieces, output periods
    ([6000, 5000], [16, 9], 32, 8, 128, 4, 16, False, torch.bfloat16),        # 64 columns, registers moved
    ([5000, 4000], [64, 20], 32, 8, 128, 4, 64, True, torch.bfloat16),        # the wide form, one half and two
    ([50] * 200, [1] * 200, 2, 2, 64, 4, 16, True, torch.bfloat16),           # whole items of one tile
]


@pytest.mark.parametrize("form", FORMS, ids=[str(i) for i in range(len(FORMS))])
def test_attention_gives_up_and_the_context_survives(c, form):
    *shape, causal, dtype = form
    q, cache, batch, _, _ = _case(c, *shape, causal, seed=77)
    want = c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dtype)
    c.mxs_sync()
    # from a limit that no first tile can meet to some that only a few waits pass, if any
    for limit in (1, 300, 1000, 3000):
        c.mxs_set_wait_limit(limit)
        try:
            got = c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dtype)
            try:
                c.mxs_sync()
                assert limit > 1 and torch.equal(got, want)
            except c.MxsError as e:
                assert e.status == MXS_ERR_TIMEOUT
        finally:
            c.mxs_set_wait_limit(0)
        c.mxs_sync()                                   # the word was cleared by the first read
        assert torch.equal(c.mxs_attn_tree(q, cache, batch, 0.1, dtype=dtype), want)
        c.mxs_sync()


def test_a_step_behind_one_that_gave_up(c):
    """Calls queued behind it on the stream, the framework's other
    tensor-core kernels among them, run as ever."""
    q, cache, batch, _, _ = _case(c, [5000, 4000], [64, 20], 32, 8, 128, 4, 64, True, seed=78)
    want = c.mxs_attn_tree(q, cache, batch, 0.1)
    x = torch.randn(256, 4096, device="cuda")
    lay = c.mxs_layout_make(4096, (0, 0, 4096))
    A, W = c.mxtensor_empty(256, lay), c.mxtensor_empty(256, lay)
    c.mxs_quantize_act(x, A)
    c.mxs_quantize_weight(x, W)
    Y = c.mxs_gemm(A, W)
    c.mxs_sync()
    c.mxs_set_wait_limit(1)
    try:
        c.mxs_attn_tree(q, cache, batch, 0.1)
    finally:
        c.mxs_set_wait_limit(0)                        # (synchronous: behind the call)
    again = [c.mxs_attn_tree(q, cache, batch, 0.1) for _ in range(3)]
    Z = c.mxs_gemm(A, W)
    with pytest.raises(c.MxsError) as e:
        c.mxs_sync()
    assert e.value.status == MXS_ERR_TIMEOUT
    assert all(torch.equal(a, want) for a in again) and torch.equal(Y, Z)
