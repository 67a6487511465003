"""q8_kv_plan when the free pages run out over a table that other sequences have used: no entry keeps an old page, and
the same step planned again with pages enough is the step."""
import numpy as np
import pytest

from . import _kv_ref as ref
from .test_kv_plan_gpu import check, expect_data_error, run, setup

pytestmark = pytest.mark.gpu

CACHED, FRESH, PAGE = [14, 31, 8], [4, 40, 20], 16


def used_table(rng):
    """A table whose entries behind each row's pages hold page ids in range, as a finished sequence left them."""
    table, free, n_pages = setup(rng, CACHED, FRESH, PAGE)
    table[table < 0] = rng.integers(0, n_pages, int((table < 0).sum()))
    return table, free, n_pages


def short_of(want, have, n_free):
    """The reference's outputs with -1 in the entries that got no page."""
    table, used = want[0].copy(), 0
    for b, (c, f) in enumerate(zip(CACHED, FRESH)):
        for i in range(have[b], ref.pages_of(c + f, PAGE)):
            if used >= n_free:
                table[b, i] = -1
            used += 1
    return (table, *want[1:])


@pytest.mark.parametrize("n_free", [0, 1, 2, 3])
def test_an_entry_without_a_page_keeps_no_old_one(q8, n_free):
    rng = np.random.default_rng(70 + n_free)
    table, free, n_pages = used_table(rng)
    held = [ref.pages_of(c, PAGE) for c in CACHED]
    total = sum(FRESH)
    want = short_of(ref.plan(CACHED, FRESH, PAGE, free[:n_free], table, total), held, n_free)
    assert want[5] > n_free
    got = run(q8, CACHED, FRESH, PAGE, free[:n_free], table, n_pages, total)
    q8.q8_check()
    check(got, want, total, total, None)
    # planned again over what the short call left, with pages enough
    again = run(q8, CACHED, FRESH, PAGE, free, got["table"], n_pages, total, held=held)
    q8.q8_check()
    check(again, ref.plan(CACHED, FRESH, PAGE, free, table, total), total, total, None)
    # held_out of the short call as `held`: the missing pages are reported, nothing gets a page of another sequence
    wrong = run(q8, CACHED, FRESH, PAGE, free, got["table"], n_pages, total, held=got["held_out"].tolist())
    expect_data_error(q8)
    assert np.array_equal(wrong["table"], got["table"]) and wrong["needed"].tolist() == [0]
    assert wrong["slots"].tolist() == want[2].tolist()


@pytest.mark.parametrize("n_free", [0, 1, 2, 3])
def test_the_next_step_goes_on_with_the_pages_that_there_are(q8, n_free):
    """What a row has is held_out less its entries of -1: with the tokens that got a slot, a step like any other."""
    rng = np.random.default_rng(80 + n_free)
    table, free, n_pages = used_table(rng)
    got = run(q8, CACHED, FRESH, PAGE, free[:n_free], table, n_pages, sum(FRESH))
    held = [int(h) - int((row[:h] == -1).sum()) for h, row in zip(got["held_out"], got["table"])]
    assert sum(held) == sum(ref.pages_of(c, PAGE) for c in CACHED) + n_free
    ends = np.cumsum(FRESH)
    cached = [c + int((got["slots"][e - f:e] >= 0).sum()) for c, f, e in zip(CACHED, FRESH, ends)]
    fresh, left = [20, 3, 1], free[n_free:]
    again = run(q8, cached, fresh, PAGE, left, got["table"], n_pages, sum(fresh), held=held)
    q8.q8_check()
    check(again, ref.plan(cached, fresh, PAGE, left, got["table"], sum(fresh), held=held), sum(fresh), sum(fresh), None)


def test_a_free_page_out_of_range_leaves_no_old_entry(q8):
    rng = np.random.default_rng(75)
    table, free, n_pages = used_table(rng)
    free = free.copy()
    free[1] = n_pages
    got = run(q8, CACHED, FRESH, PAGE, free, table, n_pages, sum(FRESH))
    expect_data_error(q8)
    assert got["table"][0, 1] == free[0] and got["table"][1, 2] == -1 and got["table"][1, 3] == free[2]
    assert (got["slots"][4:8] >= 0).sum() == 1 and (got["slots"] == -1).sum() == 16
