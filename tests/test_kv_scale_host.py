"""q8_tree_attention refuses a softmax scale that is not finite, whatever kernel the sizes choose."""
import ctypes

import pytest

import int8_quantized_projection_gb300 as q8p
from int8_quantized_projection_gb300 import build

from .test_kv_abi_host import FAKE, LONG, MISALIGNED, P, desc, ref

ERR_ARG, ERR_ALIGN = 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q8p.lib()


def attend(lib, scale, fresh, most, q=MISALIGNED):
    # the misaligned q keeps every call from the GPU
    return lib.q8_tree_attention(ref(desc()), 0, P(q), 28, ctypes.c_float(scale), P(FAKE), 4, P(FAKE), P(FAKE), 2, P(0), 64,
                                 fresh, most, P(FAKE), P(0), P(0), P(FAKE), 1 << 30, P(0))


@pytest.mark.parametrize("most", [64, LONG])
@pytest.mark.parametrize("fresh", [1, 2, 16])  # 8, 16 and 128 rows a unit
def test_scale(lib, fresh, most):
    for bad in (float("nan"), float("inf"), float("-inf"), 3e38, -3e38):
        assert attend(lib, bad, fresh, most) == ERR_ARG, bad
    for good in (0.0, -0.0, 0.088, -1.0, 1e-40, 2.3e38):
        assert attend(lib, good, fresh, most) == ERR_ALIGN, good
