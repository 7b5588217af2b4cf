"""Where the decoded values of mxs_attn_tree stop being exact: at blocks whose
largest magnitude is 2^123."""
import pytest
import torch

from tests import parity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c():
    parity.need_gpu()
    return parity.capi()


@pytest.mark.parametrize("rows", [3, 80])                            # tokens as the matrix rows; the wide form
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_largest_blocks(c, bits, d, rows):
    """One token that sees itself: the output is its decoded V."""
    B = 4
    cache = c.kv_cache_empty(B, 1, d, bits)
    g = torch.Generator(device="cuda")
    g.manual_seed(bits + d)
    x = torch.rand((B, 1, d), generator=g, device="cuda") - 0.5
    x[:, :, ::32] = 1.75                                             # the block's largest, in [1, 2)
    v = x * 2.0 ** torch.tensor([0.0, 121.0, 122.0, 123.0], device="cuda")[:, None, None]
    c.mxs_kv_write(torch.zeros_like(v), v, cache, torch.arange(B, device="cuda"))
    seg = 2 if bits == 4 else 0
    assert cache.V.scale_rows(seg)[:, 0].tolist() == [127, 248, 249, 250]
    want = c.mxs_kv_read(cache, torch.arange(B, device="cuda"), dtype=torch.float32)[1]
    want[3] /= 2                                                     # as if its scale byte were 249
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn((B, rows, d), generator=g, device="cuda").to(torch.bfloat16)
    batch = c.tree_batch(torch.arange(B + 1, **i32), torch.zeros(B, **i32), torch.arange(B, **i32)[:, None], 1, max_q=1, max_len=1)
    for dtype in (torch.float32, torch.bfloat16):
        out = c.mxs_attn_tree(q, cache, batch, 1.0, dtype=dtype)
        c.mxs_sync()
        assert torch.equal(out, want.to(dtype).expand(B, rows, d))
