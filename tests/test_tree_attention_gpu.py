"""q8_tree_attention against the definition in 64 bits, value by value, within the limit derived in _kv_ref."""
import numpy as np
import pytest

from . import _kv_ref as ref

pytestmark = pytest.mark.gpu


def trees(case, reach=8):
    out = []
    for f in case.fresh:
        out += ref.tree(case.rng, f, reach)[1]
    return out


def check(case, y, masks=None, **kw):
    want, lim = case.reference(masks, **kw)
    return ref.assert_within(y.cpu().numpy()[:case.total], want, lim)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (7, 1), (28, 4), (16, 16), (10, 2), (24, 1)])
@pytest.mark.parametrize("cached,page", [([0], 16), ([1], 16), ([15, 16, 17], 16), ([300, 0, 129], 48)])
def test_single_tokens(q8, int8, d, heads, kv_heads, cached, page):
    c = ref.Case(1, cached, [1] * len(cached), heads, kv_heads, d, page, int8)
    check(c, c.run())
    q8.q8_check()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,cached,fresh,page", [
    (128, 28, 4, [130, 7], [16, 9], 32), (64, 4, 4, [0, 250, 33], [64, 1, 40], 16), (128, 12, 1, [1000], [33], 64),
    (64, 64, 1, [77], [3], 128), (128, 2, 2, [127, 128, 129], [2, 3, 4], 16), (128, 14, 2, [5], [64], 256)])
def test_trees(q8, int8, d, heads, kv_heads, cached, fresh, page):
    c = ref.Case(2, cached, fresh, heads, kv_heads, d, page, int8)
    m = trees(c)
    check(c, c.run(m), m)
    q8.q8_check()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,cached,fresh,page", [
    (128, 4, 2, [0], [200], 16), (64, 7, 1, [100], [130], 64), (128, 28, 4, [3, 0, 50], [20, 0, 65], 32),
    (64, 2, 2, [0, 0], [1, 257], 48), (128, 3, 1, [640], [127], 128)])
def test_prompts_are_causal(q8, int8, d, heads, kv_heads, cached, fresh, page):
    c = ref.Case(3, cached, fresh, heads, kv_heads, d, page, int8)
    check(c, c.run())
    q8.q8_check()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,fresh", [(4, 1), (4, 4), (16, 5)])
def test_a_long_context_is_split_and_joined(q8, int8, heads, fresh):
    c = ref.Case(4, [9000, 4321, 17], [fresh] * 3, heads, 2, 128, 64, int8)
    m = trees(c) if fresh > 1 else None
    check(c, c.run(m), m)
    q8.q8_check()


@pytest.mark.parametrize("batch", [40, 300])
def test_ragged_batches(q8, batch):
    rng = np.random.default_rng(batch)
    c = ref.Case(5, rng.integers(0, 90, batch).tolist(), rng.integers(0, 3, batch).tolist(), 4, 2, 64, 16, False)
    m = trees(c)
    check(c, c.run(m), m)
    q8.q8_check()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,fresh", [(2, 6), (8, 30)])
def test_rows_whose_mask_leaves_nothing(q8, int8, heads, fresh):
    c = ref.Case(6, [0, 0], [fresh, fresh], heads, 1, 64, 16, int8)
    m = trees(c)
    m[0] = m[3] = m[fresh + 1] = 0
    m[2] = 1 << (fresh - 1)  # sees another node, not itself
    y, qs, ds = c.run(m, plane=True)
    check(c, y, m)
    assert (y[[0, 3, fresh + 1]] == 0).all() and (qs[[0, 3, fresh + 1]] == 0).all()
    q8.q8_check()


def test_mask_bits_past_the_fresh_tokens_see_nothing(q8):
    c = ref.Case(7, [20, 9], [3, 5], 4, 2, 64, 16, False)
    m = trees(c)
    a = c.run(m)
    full = [x | ~((1 << f) - 1) & (2 ** 64 - 1) for x, f in zip(m, [3] * 3 + [5] * 5)]
    assert c.torch.equal(a, c.run(full))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,cached,fresh", [(4, [70], [1]), (28, [200, 3], [16, 5])])
def test_plane_is_the_encoding_of_y(q8, int8, heads, cached, fresh):
    import torch

    c = ref.Case(8, cached, fresh, heads, 4, 128, 16, int8)
    y, qs, ds = c.run(plane=True)
    check(c, y)
    qr, dr = q8.empty_plane(c.total, heads * 128)
    q8.quantize_q8_0(y, qr, dr)
    assert torch.equal(qs, qr) and torch.equal(ds, dr)
    # the plane alone: the same bytes
    q2, d2 = q8.empty_plane(c.total, heads * 128)
    q8.q8_tree_attention(c.cache(), 0, c.dev(c.q), c.dev(c.table), c.dev(np.array(cached, np.int32)), c.dev(c.starts), None,
                         qs=q2, ds=d2, max_fresh=max(fresh))
    assert torch.equal(qs, q2) and torch.equal(ds, d2)
    q8.q8_check()


@pytest.mark.parametrize("heads", [4, 16])
def test_rows_behind_the_last_sequence_are_left(q8, heads):
    import torch

    c = ref.Case(9, [40, 7], [3, 2], heads, 2, 64, 16, False)
    m = trees(c)
    y, qs, ds = c.run(m, plane=True, tokens=9)
    check(c, y, m)
    assert torch.isnan(y[5:]).all() and (qs[5:] == 77).all() and (ds[5:] == 77).all()


@pytest.mark.parametrize("int8", [False, True])
def test_layers(q8, int8):
    c = ref.Case(10, [100], [4], 8, 2, 64, 16, int8, layers=3)
    for layer in range(3):
        check(c, c.run(layer=layer), layer=layer)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3])
def test_scale(q8, scale):
    c = ref.Case(11, [60], [3], 4, 2, 64, 16, False)
    want, lim = c.reference(scale=scale)
    lim_abs = c.reference(scale=abs(scale))[1]
    ref.assert_within(c.run(scale=scale).cpu().numpy(), want, np.maximum(lim, lim_abs))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e30])
def test_queries_of_any_size(q8, int8, size):
    """The row's power of two keeps tiny and huge queries exact; the scale brings the scores back."""
    c = ref.Case(12, [90], [5], 4, 2, 128, 16, int8)
    c.q = (c.q * np.float32(size)).astype(np.float32)
    c.q[0, :64] *= np.float32(1e-3)
    scale = float(np.float32(0.09 / size))
    want, lim = c.reference(scale=scale)
    ref.assert_within(c.run(scale=scale).cpu().numpy(), want, lim)


def test_value_scales_of_any_size(q8):
    """int8 scales from 1e-30 to 1e30 in one context: each row's weights follow the largest it sees."""
    c = ref.Case(13, [200, 150], [6, 4], 4, 2, 64, 16, True)
    c.vs = (10.0 ** c.rng.uniform(-30, -25, c.vs.shape)).astype(np.float32)
    c.vs[:, c.table[1, :10]] = (10.0 ** c.rng.uniform(25, 30, c.vs[:, c.table[1, :10]].shape)).astype(np.float32)
    c.v = c.vc.astype(np.float64) * c.vs[..., None]
    m = trees(c)
    want, lim = c.reference(m)
    # a weight far below the row's largest v scale loses bits against its own v, not against the sum: the limit is
    # taken on the largest |v| a row sees, one step of f16 at weight 2^-24
    worst = np.abs(c.v).max((0, 1, 2, 3, 4))
    big = np.array([np.abs(c.v[0][c.table[b, :1 + 9 * (b == 1) + 12 * (b == 0)]]).max() for b in (0, 1)])
    lim = lim + np.repeat(big, c.fresh)[:, None] * 2.0 ** -20
    assert worst > 0
    ref.assert_within(c.run(m).cpu().numpy(), want, lim)


@pytest.mark.parametrize("heads,fresh", [(4, 6), (28, 17), (64, 33)])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 65504.0])
def test_what_a_row_cannot_see_does_not_reach_it(q8, heads, fresh, bad):
    """Stale values behind the sequence and hidden nodes hold NaN, infinities or the type's largest; only rows that
    see such a node are not finite."""
    c = ref.Case(14, [37, 64], [fresh, fresh], heads, 1, 64, 16, False)
    m = [1 << i for _ in (0, 1) for i in range(fresh)]  # every node sees itself and the cached tokens
    clean = c.run(m)
    for b in (0, 1):  # everything behind the last token of the sequence's last page, and the spare pages
        n = c.cached[b] + fresh
        if n % 16:
            c.kc[:, c.table[b, n // 16], :, n % 16:] = bad
            c.vc[:, c.table[b, n // 16], :, n % 16:] = bad
    used = set(c.table[c.table >= 0].tolist())
    for p in set(range(c.kc.shape[1])) - used:
        c.kc[:, p], c.vc[:, p] = bad, bad
    assert c.torch.equal(clean, c.run(m))
    node = 3  # node 3 of both sequences
    for b in (0, 1):
        pos = c.cached[b] + node
        c.vc[:, c.table[b, pos // 16], :, pos % 16, 7] = bad
        c.kc[:, c.table[b, pos // 16], :, pos % 16, 9] = bad
    got = c.run(m)
    others = [t for t in range(2 * fresh) if t % fresh != node]
    assert c.torch.equal(clean[others], got[others])
    if not np.isfinite(bad):
        assert not c.torch.isfinite(got[[node, fresh + node]].view(2, heads, 64)[:, :, 7]).any()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_int8_scales_a_row_cannot_see_do_not_reach_it(q8, bad):
    c = ref.Case(15, [37], [6], 4, 1, 64, 16, True)
    m = [1 << i for i in range(6)]
    clean = c.run(m)
    n, node = 43, 40
    for s in (c.ks, c.vs):
        s[:, c.table[0, n // 16], :, n % 16:] = bad
        s[:, c.table[0, node // 16], :, node % 16] = bad
    got = c.run(m)
    others = [0, 1, 2, 4, 5]
    assert c.torch.equal(clean[others], got[others])
    assert not c.torch.isfinite(got[3]).any()


@pytest.mark.parametrize("heads", [2, 16])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(q8, heads):
    c = ref.Case(16, [37], [6], heads, 1, 64, 16, False)
    clean = c.run()
    c.q[2, 5], c.q[4, 64 + 1] = np.nan, np.inf
    got = c.run().view(6, heads, 64)
    spoiled = c.torch.zeros(6, heads, dtype=c.torch.bool, device="cuda")
    spoiled[2, 0] = spoiled[4, 1] = True
    assert c.torch.isnan(got[spoiled]).all()
    assert c.torch.equal(got[~spoiled], clean.view(6, heads, 64)[~spoiled])


def test_visible_non_finite_values_spoil_what_sees_them(q8):
    c = ref.Case(17, [37], [6], 4, 1, 64, 16, False)
    c.vc[0, c.table[0, 1], 0, 3, 11] = np.nan  # token 19: every row sees it
    got = c.run().view(6, 4, 64)
    assert c.torch.isnan(got[..., 11]).all()
    assert c.torch.isfinite(got[..., [i for i in range(64) if i != 11]]).all()


@pytest.mark.parametrize("what", ["cached", "starts", "fresh", "long", "pages", "page", "negative page"])
def test_a_sequence_out_of_range_is_skipped_and_reported(q8, what):
    import torch

    c = ref.Case(18, [40, 50, 60], [2, 3, 2], 4, 2, 64, 16, False)
    clean = c.run()
    kw = {}
    keep = [0, 1, 5, 6]
    if what == "cached":
        c.cached[1] = -1
    elif what == "starts":
        c.starts[3] = 9  # past the rows of q
        keep = [0, 1, 2, 3, 4]
    elif what == "fresh":
        kw["max_fresh"] = 2
    elif what == "long":
        kw["max_len"] = 52
        keep = [0, 1]
    elif what == "pages":
        c.cached[1] = 16 * c.table.shape[1]
        kw["max_len"] = 4096
    else:
        c.table[1, 2] = c.kc.shape[1] if what == "page" else -7
    got = c.run(**kw)
    with pytest.raises(q8.Q8Error) as e:
        q8.q8_check()
    assert e.value.status == 8
    q8.q8_check()
    assert torch.equal(got[keep], clean[keep])
    if "page" not in what or what == "pages":
        skipped = [r for r in range(7) if r not in keep]
        if what == "long":
            skipped = [2, 3, 4, 5, 6]
        assert torch.isnan(got[skipped]).all()


def test_results_repeat(q8):
    c = ref.Case(19, [3000, 100, 7], [5, 5, 5], 14, 2, 128, 32, False)
    m = trees(c)
    a = c.run(m)
    for _ in range(3):
        assert c.torch.equal(a, c.run(m))


def test_a_page_shared_by_two_sequences(q8):
    c = ref.Case(20, [32, 32], [1, 1], 4, 2, 64, 16, False)
    c.table[1, :2] = c.table[0, :2]
    check(c, c.run())


def test_offsets_past_32_bits(q8):
    """Pages whose elements lie past 2^31: the last pages of a cache of more than 4 GiB per matrix."""
    import torch

    pages, page, kv_heads, d = 17000, 256, 4, 128  # 2.2e9 values, 17.4e6 rows
    k = torch.zeros(1, pages, kv_heads, page, d, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    cache = q8.KvCache(k, v)
    ids = [pages - 1, 0, pages - 2]
    n = 3 * page
    slots = torch.tensor([ids[t // page] * page + t % page for t in range(n)], dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    kk, vv = (torch.randn(n, kv_heads * d, generator=g, device="cuda") for _ in range(2))
    q8.q8_kv_append(cache, 0, kk, vv, slots)
    assert torch.equal(v[0, pages - 1, 1, 5], vv[5, d:2 * d].half())
    q = torch.randn(2, 8 * d, generator=g, device="cuda")
    y = torch.empty_like(q)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q8.q8_tree_attention(cache, 0, q, i32([ids]), i32([n - 2]), i32([0, 2]), y, max_fresh=2)
    q8.q8_check()
    kd = kk.half().double().cpu().numpy().reshape(n, kv_heads, d).transpose(1, 0, 2)[None]
    vd = vv.half().double().cpu().numpy().reshape(n, kv_heads, d).transpose(1, 0, 2)[None]
    want, lim = ref.attention(q.cpu().numpy(), kd, vd, n, np.zeros((1, 1), int), [n - 2], [2], 8, d ** -0.5)
    ref.assert_within(y.cpu().numpy(), want, lim)


@pytest.mark.parametrize("heads,n", [(1, 10_300_000), (17, 800_000)])
def test_a_stretch_of_keys_longer_than_an_accumulation_chain(q8, heads, n):
    """All values near 1, so that a truncating accumulation over a CTA's whole stretch would show.  The tensor core
    loses up to 2^-23 of the running sum per MMA; over chains of 64 MMAs whose sum grows steadily that is at most
    64 / 2 * 2^-23 = 2^-18, and as much for scores, weights and the quotient."""
    import torch

    g = torch.Generator("cuda").manual_seed(3)
    page, d = 256, 64
    pages = ref.pages_of(n, page)
    k = torch.empty(1, pages, 1, page, d, dtype=torch.float16, device="cuda").normal_(generator=g)
    v = torch.empty_like(k).normal_(generator=g).mul_(0.25).add_(1.0)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(1, -1)
    q = torch.randn(1, heads * d, generator=g, device="cuda")
    y = torch.empty_like(q)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q8.q8_tree_attention(q8.KvCache(k, v), 0, q, table, i32([n - 1]), i32([0, 1]), y, max_fresh=1)
    q8.q8_check()
    kk, vv = (x[0, table[0].long(), 0].reshape(-1, d)[:n] for x in (k, v))
    for h in range(heads):
        p = torch.softmax(kk.double() @ q[0, h * d:(h + 1) * d].double() * d ** -0.5, 0)
        want = p @ vv.double()
        rel = ((y[0, h * d:(h + 1) * d].double() - want).abs() / want.abs()).max().item()
        assert rel <= 2.0 ** -17, (h, rel)
