"""The norm-wise limit of the attention tests tells two f16 parts from one (planted in the 64-bit reference, on the CPU)."""
import pytest

from . import _kv_norm as norm
from . import _kv_ref as ref
from ._kv_norm_cases import CASES, build


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("name", [n for n, c in CASES.items() if max(c["cached"]) < 3000])
def test_one_part_is_past_the_limit(name, int8):
    case, masks = build(name, int8)
    want, size = norm.attention(case, masks)
    plain, lim = case.reference(masks)
    ref.assert_within(want.reshape(case.total, -1), plain, lim)
    two = norm.error(norm.attention(case, masks, 2, 2)[0], want, size)
    assert two <= norm.LIMIT / 8
    assert norm.error(norm.attention(case, masks, 1, 2)[0], want, size) >= 4 * norm.LIMIT
    assert norm.error(norm.attention(case, masks, 2, 1)[0], want, size) >= 4 * norm.LIMIT
