"""rmsnorm_residual_quant's ring over many rows at widths where it has few slots, down to one, and up to 19 vectors a row."""
import numpy as np
import pytest

from tests.test_residual_norm_gpu import call, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [544, 800, 2080, 4096, 4128, 5120, 7168, 8192])
@pytest.mark.parametrize("top_k,dense,post,gate", [(0, True, True, "row"), (1, True, False, "channel"), (2, False, True, "none"),
                                                   (16, True, True, "row")])
def test_ring(q8, d, top_k, dense, post, gate):
    rows = 333 if top_k < 16 else 160
    a = inputs(np.random.default_rng([d, top_k]), rows, d, top_k, dense, post, gate)
    got = call(q8, a, pad=5)
    check(a, got)
    again = call(q8, a, pad=5, in_place=True)
    for one, other in zip(got, again):
        assert np.array_equal(one, other)
