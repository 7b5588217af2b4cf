"""The serving calls without the binding's extension: the same bits, and the
same refusals."""
import pytest
import torch

from tests import parity
from tests.test_gpu_serving import _case, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c():
    parity.need_gpu()
    return parity.capi()


def test_without_the_extension(c, monkeypatch):
    q, cache, batch, _, _ = _case(c, [500, 260], [8, 5], 8, 2, 128, 4, 16, False, seed=17)
    plan, pos, slot = c.mxs_rope_plan(128), torch.arange(13, device="cuda") + 5000, torch.arange(13, device="cuda")
    k, v = (_randn(13, 2, 128, seed=i, dtype=torch.bfloat16) for i in (1, 2))

    def calls():
        other = c.kv_cache_empty(13, 2, 128, 8)
        r = c.mxs_rope(q, pos, plan, dtype=torch.float32)
        c.mxs_kv_write(k, v, other, slot, pos=pos, rope=plan)
        a = c.mxs_attn_tree(q, cache, batch, 0.1, return_lse=True)
        b = c.mxs_attn_tree(q, cache, batch, 0.1, dtype=torch.float32, workspace=c.attn_tree_workspace(q, cache, batch))
        with pytest.raises(c.MxsError) as e:
            c.mxs_rope(q, pos, c.mxs_rope_plan(256))
        assert e.value.status == 2
        return [r, *c.mxs_kv_read(other, slot), *a, b]
    assert c._binding is not None
    want = calls()
    monkeypatch.setattr(c, "_binding", None)
    got = calls()
    c.mxs_sync()
    assert len(got) == len(want) and all(torch.equal(x, y) for x, y in zip(got, want))
