"""q8_kv_plan against a plain loop: starts, pages, slots, positions and ancestor masks are whole numbers and equal."""
import numpy as np
import pytest

from . import _kv_ref as ref

pytestmark = pytest.mark.gpu


def run(q8, cached, fresh, page, free, table, n_pages, tokens, parents=None, held=None, **kw):
    import torch

    dev = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(np.asarray(a, t))).cuda()  # noqa: E731
    b = len(cached)
    out = dict(table=dev(table), starts=torch.full((b + 1,), -7, dtype=torch.int32, device="cuda"),
               slots=torch.full((tokens,), -7, dtype=torch.int32, device="cuda"),
               positions=torch.full((tokens,), -7, dtype=torch.int32, device="cuda"),
               needed=torch.full((1,), -7, dtype=torch.int32, device="cuda"),
               held_out=torch.full((b,), -7, dtype=torch.int32, device="cuda"),
               masks=torch.full((tokens,), -7, dtype=torch.int64, device="cuda") if parents is not None else None)
    par = None
    if parents is not None:
        par = np.zeros(tokens, np.int32)
        par[:len(parents)] = parents
    q8.q8_kv_plan(dev(cached), dev(fresh), dev(free) if len(free) else None, out["table"], page, n_pages, out["starts"],
                  out["slots"], out["positions"], out["needed"], parents=None if par is None else dev(par),
                  masks=out["masks"], held=None if held is None else dev(held), held_out=out["held_out"], **kw)
    return {k: v.cpu().numpy() if v is not None else None for k, v in out.items()}


def setup(rng, cached, fresh, page, held=None, spare=4):
    b = len(cached)
    width = max(max(ref.pages_of(c + f, page) for c, f in zip(cached, fresh)), max(held or [0]), 1) + 1
    have = held or [ref.pages_of(c, page) for c in cached]
    need = sum(have) + sum(ref.pages_of(c + f, page) for c, f in zip(cached, fresh)) + spare
    ids = rng.permutation(need).astype(np.int32)
    table = np.full((b, width), -1, np.int32)
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, ids[at:], need


def check(got, want, total, tokens, parents):
    table, starts, slots, positions, masks, needed, held_out = want
    assert got["starts"].tolist() == starts
    assert got["needed"].tolist() == [needed]
    assert got["held_out"].tolist() == held_out
    assert np.array_equal(got["table"], table)
    assert got["slots"].tolist() == slots.tolist()
    assert got["positions"][:total].tolist() == [positions[t] for t in range(total)]
    assert (got["positions"][total:] == -7).all(), "positions behind the last sequence were written"
    if parents is not None:
        assert np.array_equal(got["masks"][:total], ref.as_i64([masks[t] for t in range(total)]))
        assert (got["masks"][total:] == -7).all(), "masks behind the last sequence were written"


@pytest.mark.parametrize("batch,most_cached,most_fresh,page,pad", [
    (1, 0, 1, 16, 0), (1, 100, 1, 16, 0), (1, 63, 2, 64, 3), (3, 40, 7, 16, 5), (31, 500, 9, 48, 0), (32, 500, 9, 32, 1),
    (33, 500, 64, 16, 0), (100, 3000, 33, 128, 40), (1025, 90, 5, 16, 0), (4096, 700, 3, 64, 100), (1, 17, 5000, 16, 11),
    (2, 0, 70000, 256, 0)])
def test_chain(q8, batch, most_cached, most_fresh, page, pad):
    rng = np.random.default_rng(batch * 1000 + most_fresh)
    cached = rng.integers(0, most_cached + 1, batch).tolist()
    fresh = rng.integers(0, most_fresh + 1, batch).tolist()
    cached[-1], fresh[0] = most_cached, most_fresh
    table, free, n_pages = setup(rng, cached, fresh, page)
    total = sum(fresh)
    got = run(q8, cached, fresh, page, free, table, n_pages, total + pad)
    q8.q8_check()
    check(got, ref.plan(cached, fresh, page, free, table, total + pad), total, total + pad, None)


@pytest.mark.parametrize("batch,nodes", [(1, 1), (1, 2), (2, 33), (5, 64), (32, 17), (70, 64)])
@pytest.mark.parametrize("reach", [1, 8, 64])
def test_tree(q8, batch, nodes, reach):
    rng = np.random.default_rng(batch * 100 + nodes + reach)
    cached = rng.integers(0, 300, batch).tolist()
    fresh = rng.integers(0, nodes + 1, batch).tolist()
    fresh[0] = nodes
    parents = sum((ref.tree(rng, f, reach)[0] for f in fresh), [])
    table, free, n_pages = setup(rng, cached, fresh, 16)
    total = sum(fresh)
    got = run(q8, cached, fresh, 16, free, table, n_pages, total + 3, parents)
    q8.q8_check()
    check(got, ref.plan(cached, fresh, 16, free, table, total + 3, parents), total, total + 3, parents)


def test_a_chain_written_as_a_tree_has_causal_masks(q8):
    rng = np.random.default_rng(5)
    table, free, n_pages = setup(rng, [10], [64], 16)
    got = run(q8, [10], [64], 16, free, table, n_pages, 64, list(range(-1, 63)))
    assert np.array_equal(got["masks"], ref.as_i64([(2 << i) - 1 for i in range(64)]))
    assert got["positions"].tolist() == list(range(10, 74))


def test_pages_held_beyond_the_cached_tokens_are_used_first(q8):
    rng = np.random.default_rng(6)
    cached, fresh, held = [5, 16, 0, 33], [40, 1, 16, 10], [2, 3, 0, 3]
    table, free, n_pages = setup(rng, cached, fresh, 16, held)
    got = run(q8, cached, fresh, 16, free, table, n_pages, sum(fresh), held=held)
    q8.q8_check()
    check(got, ref.plan(cached, fresh, 16, free, table, sum(fresh), held=held), sum(fresh), sum(fresh), None)


@pytest.mark.parametrize("n_free", [0, 1, 3])
def test_free_pages_that_run_out(q8, n_free):
    rng = np.random.default_rng(7)
    cached, fresh = [14, 31, 8], [4, 40, 20]
    table, free, n_pages = setup(rng, cached, fresh, 16)
    free = free[:n_free]
    got = run(q8, cached, fresh, 16, free, table, n_pages, sum(fresh))
    q8.q8_check()  # running out is told by `needed`, not an error
    want = ref.plan(cached, fresh, 16, free, table, sum(fresh))
    check(got, want, sum(fresh), sum(fresh), None)
    assert got["needed"][0] > n_free and (got["slots"] == -1).any()


def test_running_it_again_writes_the_same(q8):
    rng = np.random.default_rng(8)
    cached, fresh = [14, 31, 8], [4, 40, 20]
    table, free, n_pages = setup(rng, cached, fresh, 16)
    a = run(q8, cached, fresh, 16, free, table, n_pages, sum(fresh))
    b = run(q8, cached, fresh, 16, free, a["table"], n_pages, sum(fresh))
    for k in a:
        assert a[k] is None or np.array_equal(a[k], b[k]), k


def expect_data_error(q8):
    with pytest.raises(q8.Q8Error) as e:
        q8.q8_check()
    assert e.value.status == 8
    q8.q8_check()  # reported once


@pytest.mark.parametrize("what", ["cached", "fresh", "overflow", "held", "table", "wide", "free", "tokens", "nodes",
                                  "parent", "later parent"])
def test_values_out_of_range_are_reported_and_cost_only_their_sequence(q8, what):
    rng = np.random.default_rng(9)
    cached, fresh, page = [20, 30, 40], [3, 5, 4], 16
    table, free, n_pages = setup(rng, cached, fresh, page)
    tokens, parents, held = 12, None, None
    if what == "cached":
        cached[1] = -4
    elif what == "fresh":
        fresh[1] = -2
    elif what == "overflow":
        cached[1] = 2 ** 31 - 3
    elif what == "held":
        held = [2, 1, 3]  # 30 cached tokens need two pages
    elif what == "table":
        table[1, 1] = n_pages + 9
    elif what == "wide":
        cached[1] = 16 * table.shape[1]
    elif what == "free":
        free[0] = n_pages
    elif what == "tokens":
        tokens = 9
    elif what == "nodes":
        fresh[1] = 65
        tokens = 72
        table, free, n_pages = setup(rng, cached, fresh, page)
        parents = [-1] * 72
    elif what == "parent":
        parents = [-1, 0, 1] + [-1, 0, 3, 2, 1] + [-1, 0, 1, 2]
        parents[3 + 2] = 2  # a node is not its own parent
    else:
        parents = [-1, 0, 1] + [-2, 0, 1, 2, 1] + [-1, 0, 1, 2]
    got = run(q8, cached, fresh, page, free, table, n_pages, tokens, parents, held)
    expect_data_error(q8)
    # the first sequence is planned as ever
    want = ref.plan(cached[:1], fresh[:1], page, free, table[:1], 3, parents[:3] if parents else None)
    if what != "free":
        assert got["slots"][:3].tolist() == want[2].tolist()
    if what in ("nodes", "parent", "later parent"):
        bad = slice(3, 3 + fresh[1])
        assert (got["masks"][bad] == 0).all() and got["masks"][0] == 1
    if what in ("held", "wide", "overflow", "nodes"):
        assert (got["slots"][3:3 + fresh[1]] == -1).all()
    if what == "table":
        assert (got["slots"][3:8] == [s if p // page != 1 else -1 for s, p in zip(got["slots"][3:8], range(30, 35))]).all()
