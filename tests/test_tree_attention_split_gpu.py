"""Both ways of sharing the units among CTAs, a cluster (128 rows: a CTA) per unit and the line of all units, on the same
inputs: the host's bound on the lengths chooses (a large one the line)."""
import numpy as np
import pytest

from . import _kv_ref as ref
from .test_tree_attention_gpu import check, trees

pytestmark = pytest.mark.gpu

LINE = 1 << 20  # a bound far above the lengths


def both(case, masks=None, **kw):
    """y of either form, each within the limit; the forms' results."""
    out = []
    for most in (max(c + f for c, f in zip(case.cached, case.fresh)), LINE // case.page * case.page):
        case.table = np.pad(case.table, ((0, 0), (0, max(0, most // case.page + 1 - case.table.shape[1]))), constant_values=-1)
        y = case.run(masks, max_len=most, **kw)
        check(case, y, masks)
        out.append(y)
    case.q8.q8_check()
    return out


def clusters(q8, case, most):
    return not q8.q8_tree_attention_needs_workspace(case.cache(), case.heads, len(case.cached), max(case.fresh), most)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads", [(128, 28, 4), (64, 8, 1), (128, 12, 1), (64, 32, 2)])
@pytest.mark.parametrize("cached", [[0], [1, 0], [190, 191, 192, 193], [1000], [1400, 3, 700, 0, 15]])
def test_single_tokens(q8, int8, d, heads, kv_heads, cached):
    c = ref.Case(100, cached, [1] * len(cached), heads, kv_heads, d, 16, int8)
    assert clusters(q8, c, max(cached) + 1) and not clusters(q8, c, LINE)
    both(c)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,fresh", [(2, [3, 2]), (4, [4, 1]), (1, [8]), (7, [2, 0, 1])])
def test_small_trees_and_chains(q8, int8, heads, fresh):
    cached = [700, 20, 5][:len(fresh)]
    c = ref.Case(101, cached, fresh, heads, 1, 128, 32, int8)
    both(c)
    m = trees(c)
    both(c, m)
    m[0] = 0  # sees nothing of the tree
    both(c, m)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,cached,fresh", [
    (128, 28, 4, [380], [16]), (128, 28, 4, [100, 0, 128], [3, 5, 0]), (64, 8, 2, [700, 0], [33, 64]), (64, 64, 1, [5], [1])])
def test_units_of_128_rows(q8, int8, d, heads, kv_heads, cached, fresh):
    c = ref.Case(107, cached, fresh, heads, kv_heads, d, 16, int8)
    assert clusters(q8, c, max(a + b for a, b in zip(cached, fresh)))
    both(c)
    m = trees(c)
    both(c, m)
    m[0] = 0
    both(c, m)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("cached,fresh", [([0], [300]), ([130, 0], [70, 129])])
def test_prompts(q8, int8, cached, fresh):
    c = ref.Case(108, cached, fresh, 14, 2, 128, 32, int8)
    assert clusters(q8, c, 300)
    both(c)


@pytest.mark.parametrize("batch", [1, 14, 15, 34, 35, 74, 75, 152, 153])
def test_any_number_of_units(q8, batch):
    """8, 4, 2 and 1 CTAs a unit, and the line."""
    rng = np.random.default_rng(batch)
    cached = rng.integers(0, 900, batch)
    cached[0] = 1000
    fresh = np.where(rng.random(batch) < 0.9, 1, 0)
    fresh[0] = 1
    c = ref.Case(102, cached.tolist(), fresh.tolist(), 2, 1, 64, 16, False)
    assert clusters(q8, c, 1001) == (batch <= 152)
    both(c)


@pytest.mark.parametrize("heads,fresh", [(4, 1), (16, 1), (20, 2)])
def test_more_units_than_ctas(q8, heads, fresh):
    """8, 16 and 128 rows a unit, dealt out to CTAs; empty sequences among them."""
    rng = np.random.default_rng(heads)
    f = rng.integers(0, fresh + 1, 400)
    f[0] = fresh
    c = ref.Case(109, rng.integers(0, 90, 400).tolist(), f.tolist(), heads, 1, 64, 16, False)
    assert clusters(q8, c, 92)
    both(c)
    m = trees(c)
    both(c, m)


def test_sequences_out_of_range_among_clusters(q8):
    """Skipped and reported, in either form; the others are computed."""
    for heads in (4, 16, 40):
        for most in (64, LINE):
            c = ref.Case(110, [20, 30, 10], [1, 1, 1], heads, 1, 64, 16, False)
            c.table = np.pad(c.table, ((0, 0), (0, most // 16)), constant_values=-1)
            want, lim = c.reference()
            c.cached[1] = -5
            y = c.run(max_len=most).cpu().numpy()
            with pytest.raises(q8.Q8Error):
                q8.q8_check()
            assert np.isnan(y[1]).all()
            ref.assert_within(y[[0, 2]], want[[0, 2]], lim[[0, 2]])


@pytest.mark.parametrize("int8", [False, True])
def test_plane_and_rows_that_see_nothing(q8, int8):
    import torch

    c = ref.Case(103, [0, 0], [3, 5], 2, 1, 64, 16, int8)
    m = trees(c)
    m[0] = m[4] = 0
    for most in (5, LINE):
        c.table = np.pad(c.table, ((0, 0), (0, most // 16)), constant_values=-1)
        y, qs, ds = c.run(m, plane=True, max_len=most)
        check(c, y, m)
        assert (y[[0, 4]] == 0).all() and (qs[[0, 4]] == 0).all()
        qr, dr = q8.empty_plane(c.total, 128)
        q8.quantize_q8_0(y, qr, dr)
        assert torch.equal(qs, qr) and torch.equal(ds, dr)
    q8.q8_check()


@pytest.mark.parametrize("heads,fresh", [(4, 2), (2, 8), (16, 9)])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_what_a_row_cannot_see_does_not_reach_it(q8, heads, fresh, bad):
    """Non-finite values in a node that others do not see, in either form."""
    for most in (None, LINE):
        c = ref.Case(104, [50], [fresh], heads, 1, 64, 16, False)
        m = [1 << i for i in range(fresh)]  # every node sees itself only, beside the cached tokens
        pos = 50 + fresh - 1
        c.vc[0, c.table[0, pos // 16], 0, pos % 16, 5] = bad
        if most:
            c.table = np.pad(c.table, ((0, 0), (0, most // 16 + 1 - c.table.shape[1])), constant_values=-1)
        y = c.run(m, **({"max_len": most} if most else {})).cpu().numpy()
        want, lim = c.reference(m)
        ref.assert_within(y[:-1], want[:-1], lim[:-1])
        last = y[-1].reshape(heads, 64)
        assert not np.isfinite(last[:, 5]).any() and np.isfinite(np.delete(last, 5, 1)).all()


def test_repeats_and_graph(q8):
    import torch

    c = ref.Case(105, [1000, 300], [2, 1], 14, 2, 128, 16, True)
    y = both(c)[0]
    dev = [c.dev(x) for x in (c.q, c.table, np.array(c.cached, np.int32), c.starts)]
    out, cache = torch.empty_like(y), c.cache()
    call = lambda s=None: q8.q8_tree_attention(cache, 0, *dev, out, max_fresh=2, max_len=1002, stream=s)  # noqa: E731
    call()
    assert torch.equal(out, y)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        call(s)
    out.zero_()
    g.replay()
    assert torch.equal(out, y)


def test_a_short_workspace_is_refused_where_one_is_needed(q8):
    import torch

    c = ref.Case(106, [20], [1], 4, 1, 64, 16, False)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    check(c, c.run(workspace=small))  # not needed
    c.table = np.pad(c.table, ((0, 0), (0, LINE // 16)), constant_values=-1)
    with pytest.raises(q8.Q8Error):
        c.run(workspace=small, max_len=LINE)
