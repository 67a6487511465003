"""q8_tree_attention called without bounds: the defaults hold for every batch that the call may get."""
import numpy as np
import pytest

from . import _kv_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("fresh", [[1], [64], [30, 34], [64, 1], [40, 0, 64, 33]])
def test_no_bounds(q8, int8, masked, fresh):
    import torch

    c = ref.Case(130, [17, 200, 3, 60][:len(fresh)], fresh, 4, 2, 64, 16, int8)
    m = sum((ref.tree(c.rng, f)[1] for f in fresh), []) if masked else None
    y = torch.full((c.total, 4 * 64), float("nan"), device="cuda")
    q8.q8_tree_attention(c.cache(), 0, c.dev(c.q), c.dev(c.table), c.dev(np.array(c.cached, np.int32)), c.dev(c.starts), y,
                         masks=c.dev(ref.as_i64(m)) if masked else None)
    q8.q8_check()
    want, lim = c.reference(m)
    ref.assert_within(y.cpu().numpy(), want, lim)
