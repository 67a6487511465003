"""What q8_kv_plan leaves for a draft tree that it refuses: no slots, and masks that let no token see another."""
import numpy as np
import pytest

from . import _kv_ref as ref
from .test_kv_plan_gpu import expect_data_error, run, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["cached", "overflow", "held", "wide", "many", "parent"])
@pytest.mark.parametrize("nodes", [1, 5, 40, 64])
def test_a_refused_tree_has_no_masks(q8, what, nodes):
    rng = np.random.default_rng(nodes)
    cached, fresh, page = [20, 30, 40], [3, nodes, 4], 16
    table, free, n_pages = setup(rng, cached, fresh, page)
    parents = sum((ref.tree(rng, f)[0] for f in fresh), [])
    held = [ref.pages_of(c, page) for c in cached]
    slots_kept = what == "parent"
    if what == "cached":
        cached[1] = -4
    elif what == "overflow":
        cached[1] = 2 ** 31 - 1
    elif what == "held":
        held[1] = 1  # 30 cached tokens need two pages
    elif what == "wide":
        cached[1] = 16 * table.shape[1]
        held[1] = table.shape[1]
    elif what == "many":
        held[1] = table.shape[1] + 1
    else:
        parents[3] = 0  # the first node has no node before it
    total = sum(fresh)
    got = run(q8, cached, fresh, page, free, table, n_pages, total + 2, parents, held)
    expect_data_error(q8)
    mine, behind = slice(3, 3 + nodes), slice(3 + nodes, total)
    assert (got["masks"][mine] == 0).all()
    assert ((got["slots"][mine] >= 0) == slots_kept).all()
    # the sequences around it are planned as ever
    want = ref.plan([20, 30, 40], fresh, page, free, table, total, [p if i != 3 else -1 for i, p in enumerate(parents)])
    for at in (slice(0, 3), behind):
        assert np.array_equal(got["masks"][at], ref.as_i64([want[4][t] for t in range(at.start, at.stop)]))
        assert got["positions"][at].tolist() == [want[3][t] for t in range(at.start, at.stop)]
    assert got["starts"].tolist() == want[1]
    assert got["slots"][:3].tolist() == want[2][:3].tolist() and (got["slots"][behind] >= 0).all()
