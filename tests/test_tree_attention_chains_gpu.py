"""q8_tree_attention where a unit's place on the line is searched over more than 32 row tiles, and where a piece is long
enough for its accumulator to be added to the earlier ones more than once, with scales that rise meanwhile."""
import numpy as np
import pytest

from . import _kv_norm as norm
from . import _kv_ref as ref
from .test_tree_attention_gpu import trees
from .test_tree_attention_split_gpu import LINE, clusters

pytestmark = pytest.mark.gpu

TILE = 128  # keys of a tile of the 128-row kernel
CHAIN = 4   # tiles whose products one accumulator takes


def check(case, most, masks=None):
    table = case.table
    case.table = np.pad(table, ((0, 0), (0, max(0, most // case.page + 1 - table.shape[1]))), constant_values=-1)
    y = case.run(masks, max_len=most).cpu().numpy()
    case.table = table
    case.q8.q8_check()
    want, lim = case.reference(masks)
    ref.assert_within(y, want, lim)
    exact, size = norm.attention(case, masks)
    assert norm.error(y, exact, size) <= norm.LIMIT


@pytest.mark.parametrize("int8,d", [(False, 64), (True, 64), (False, 128), (True, 128)])
@pytest.mark.parametrize("cached,fresh", [([300], [700]), ([0, 40], [5, 640])])
def test_a_prompt_of_many_row_tiles(q8, int8, d, cached, fresh):
    """A chunk whose packed rows make 35 or 39 tiles, behind cached tokens."""
    c = ref.Case(150, cached, fresh, 7, 1, d, 32, int8)
    assert max(fresh) * 7 > 32 * 128
    check(c, LINE)


def rising(case):
    """Scales of a sequence's keys and values grow with the position: each chain has other references than the last."""
    for b, (n, f) in enumerate(zip(case.cached, case.fresh)):
        pos = np.arange(n + f)
        pg, off = case.table[b][pos // case.page], pos % case.page
        grow = 2.0 ** (9 * pos / (n + f))
        if case.ks is None:
            case.kc[0, pg, :, off] *= (0.5 + pos / (n + f))[:, None, None].astype(np.float16)
            case.vc[0, pg, :, off] *= grow[:, None, None].astype(np.float16)
        else:
            case.ks[0, pg, :, off] *= (0.5 + pos / (n + f))[:, None].astype(np.float32)
            case.vs[0, pg, :, off] *= grow[:, None].astype(np.float32)
    if case.ks is None:
        case.k, case.v = case.kc.astype(np.float64), case.vc.astype(np.float64)
    else:
        case.k = case.kc.astype(np.float64) * case.ks[..., None]
        case.v = case.vc.astype(np.float64) * case.vs[..., None]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_chains_of_a_whole_unit(q8, int8, d):
    """Units of up to 16 tiles that a CTA does whole: up to three sums."""
    rng = np.random.default_rng(d)
    c = ref.Case(151, rng.integers(1200, 1990, 80).tolist(), [17] * 80, 1, 1, d, 64, int8)
    c.cached[3] = 2000
    c = ref.Case(151, c.cached, c.fresh, 1, 1, d, 64, int8)
    rising(c)
    most = max(n + f for n, f in zip(c.cached, c.fresh))
    assert clusters(q8, c, most) and (most - 1) // TILE >= 3 * CHAIN
    check(c, most, trees(c))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_chains_of_a_piece_of_the_line(q8, int8, d):
    """Two long units each shared by half the CTAs: pieces of 13 tiles, joined over the line."""
    c = ref.Case(152, [130000], [9], 4, 2, d, 128, int8)
    rising(c)
    pieces = 2 * (130000 // TILE) / 152
    assert not clusters(q8, c, LINE) and pieces > 3 * CHAIN
    check(c, LINE, trees(c))
