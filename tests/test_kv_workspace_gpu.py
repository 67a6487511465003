"""q8_tree_attention after a refused call with the same heads and bounds: the workspace is allocated as ever."""
import numpy as np
import pytest

from . import _kv_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [6, 20])
def test_a_call_behind_a_refused_one(q8, heads):
    import torch

    c = ref.Case(120 + heads, [300], [1], heads, 1, 64, 16, False)
    most = (1 << 20) + heads  # the line form, with bounds of this test's own
    c.table = np.pad(c.table, ((0, 0), (0, most // 16)), constant_values=-1)
    k = torch.zeros(1, 4, 1, 8, 64, dtype=torch.float16, device="cuda")  # pages of 8 tokens
    y = torch.zeros(1, heads * 64, device="cuda")
    args = c.dev(c.q), c.dev(c.table), c.dev(np.array(c.cached, np.int32)), c.dev(c.starts), y
    with pytest.raises(q8.Q8Error) as e:
        q8.q8_tree_attention(q8.KvCache(k, k), 0, *args, max_fresh=1, max_len=most)
    assert e.value.status == 1
    q8.q8_tree_attention(c.cache(), 0, *args, max_fresh=1, max_len=most)
    q8.q8_check()
    want, lim = c.reference()
    ref.assert_within(y.cpu().numpy(), want, lim)
