"""q8_tree_attention against 64 bits in the norm: far tighter than the limits value by value, so that a lost half of a
weight or of q shows (test_kv_norm_limit.py plants one in the reference)."""
import numpy as np
import pytest

from . import _kv_norm as norm
from ._kv_norm_cases import CASES, build

pytestmark = pytest.mark.gpu

LINE = 1 << 20  # a bound far above the lengths: units share one line


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_norm(q8, name, int8):
    case, masks = build(name, int8)
    want, size = norm.attention(case, masks)
    case.table = np.pad(case.table, ((0, 0), (0, LINE // case.page)), constant_values=-1)
    errors = {most: norm.error(case.run(masks, max_len=most).cpu().numpy(), want, size)
              for most in (max(c + f for c, f in zip(case.cached, case.fresh)), LINE)}
    q8.q8_check()
    print(f"{name} {'int8' if int8 else 'f16'}: " + ", ".join(f"{e:.2e}" for e in errors.values()))
    assert max(errors.values()) <= norm.LIMIT, errors
