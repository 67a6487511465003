"""q8_kv_append and q8_kv_accept: what lands in the cache equals the definition bit for bit, and nothing else changes."""
import numpy as np
import pytest

from . import _kv_ref as ref

pytestmark = pytest.mark.gpu


def encode(x):
    """int8 codes and f32 scale of rows, in f32 steps: d = amax / 127, q = rint(x * (1 / d))."""
    amax = np.abs(x).max(-1)
    d = (amax / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
    return np.clip(np.rint(x * inv[..., None]), -127, 127).astype(np.int8), d


def new_cache(q8, rng, layers, n_pages, kv_heads, page, d, int8):
    import torch

    shape = (layers, n_pages, kv_heads, page, d)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    if int8:
        host = [rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2)]
        host += [rng.uniform(0.01, 0.1, shape[:-1]).astype(np.float32) for _ in range(2)]
    else:
        host = [rng.normal(0, 1, shape).astype(np.float16) for _ in range(2)] + [None, None]
    return host, q8.KvCache(*[None if h is None else dev(h) for h in host])


def tensors(cache):
    return [None if t is None else t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def equal(a, b):
    return a is None or np.array_equal(a.view(np.uint8), b.view(np.uint8))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,kv_heads,page", [(1, 1, 16), (1, 4, 16), (2, 3, 48), (17, 4, 64), (333, 8, 32), (1000, 5, 128)])
def test_append(q8, int8, d, tokens, kv_heads, page):
    import torch

    rng = np.random.default_rng(tokens + d)
    n_pages = ref.pages_of(tokens, page) + 2
    host, cache = new_cache(q8, rng, 2, n_pages, kv_heads, page, d, int8)
    k, v = (rng.normal(0, 2, (tokens, kv_heads, d)).astype(np.float32) for _ in range(2))
    k[0, 0] = 0.0
    v[-1, -1, 3] = 300.0
    slots = rng.permutation(n_pages * page)[:tokens].astype(np.int32)
    if tokens > 2:
        slots[1] = -1
        slots[tokens // 2] = -5
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    q8.q8_kv_append(cache, 1, dev(k.reshape(tokens, -1)), dev(v.reshape(tokens, -1)), dev(slots))
    q8.q8_check()
    for x, c, s in ((k, 0, 2), (v, 1, 3)):
        for t in range(tokens):
            if slots[t] < 0:
                continue
            at = (1, slots[t] // page, slice(None), slots[t] % page)
            if int8:
                host[c][at], host[s][at] = encode(x[t])
            else:
                host[c][at] = x[t].astype(np.float16)
    for a, b in zip(host, tensors(cache)):
        assert equal(a, b)


@pytest.mark.parametrize("int8", [False, True])
def test_append_reports_slots_past_the_cache(q8, int8):
    import torch

    rng = np.random.default_rng(3)
    host, cache = new_cache(q8, rng, 1, 2, 2, 16, 64, int8)
    x = torch.randn(3, 128, device="cuda")
    q8.q8_kv_append(cache, 0, x, x, torch.tensor([32, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda"))
    with pytest.raises(q8.Q8Error) as e:
        q8.q8_check()
    assert e.value.status == 8
    for a, b in zip(host, tensors(cache)):
        assert equal(a, b)


def test_append_of_non_finite_rows(q8):
    """f16: stored as they are (f32 past 65504 becomes infinite); int8: the row's scale is non-finite, other rows keep theirs."""
    import torch

    x = torch.ones(4, 128, device="cuda")
    x[0, 5], x[1, 70], x[2, 0] = float("nan"), float("inf"), 70000.0
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    f = q8.empty_kv_cache(1, 1, 2, 16, 64)
    f.k.zero_(), f.v.zero_()
    q8.q8_kv_append(f, 0, x, x, slots)
    want = x.view(4, 2, 64).half().transpose(0, 1)
    assert torch.equal(torch.nan_to_num(f.k[0, 0, :, :4], 9.0), torch.nan_to_num(want, 9.0))
    i = q8.empty_kv_cache(1, 1, 2, 16, 64, int8=True)
    q8.q8_kv_append(i, 0, x, x, slots)
    s = i.k_scale[0, 0, :, :4].cpu().numpy()
    assert np.isnan(s[0, 0]) and np.isinf(s[1, 1])
    assert s[1, 0] == np.float32(1) / np.float32(127) and s[0, 1] == s[1, 0]
    assert torch.isfinite(i.v_scale[0, 0, :, 2:4]).all()
    q8.q8_check()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,kv_heads,page,layers,batch,most", [
    (64, 1, 16, 1, 1, 1), (128, 4, 16, 3, 2, 5), (128, 2, 48, 2, 7, 16), (64, 3, 64, 4, 5, 64), (128, 8, 32, 1, 40, 33)])
def test_accept(q8, int8, d, kv_heads, page, layers, batch, most):
    import torch

    rng = np.random.default_rng(d + batch)
    cached = rng.integers(0, 70, batch).tolist()
    fresh = rng.integers(0, most + 1, batch).tolist()
    fresh[0] = most
    need = [ref.pages_of(c + f, page) for c, f in zip(cached, fresh)]
    n_pages = sum(need) + 2
    ids = rng.permutation(n_pages)
    table = np.full((batch, max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    counts = np.array([rng.integers(0, f + 1) for f in fresh], np.int32)
    counts[0] = most
    paths = np.full((batch, most), -9, np.int32)
    for b, (n, f) in enumerate(zip(counts, fresh)):
        paths[b, :n] = np.sort(rng.permutation(f)[:n])
    host, cache = new_cache(q8, rng, layers, n_pages, kv_heads, page, d, int8)
    lens = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    q8.q8_kv_accept(cache, dev(table), dev(cached), dev(fresh), dev(paths), dev(counts), lens)
    q8.q8_check()
    for x in host:
        if x is None:
            continue
        old = x.copy()
        for b in range(batch):
            for j in range(counts[b]):
                s, t = cached[b] + paths[b, j], cached[b] + j
                x[:, table[b, t // page], :, t % page] = old[:, table[b, s // page], :, s % page]
    for a, b in zip(host, tensors(cache)):
        assert equal(a, b)
    assert lens.cpu().tolist() == [c + int(n) for c, n in zip(cached, counts)]


@pytest.mark.parametrize("what", ["order", "past", "negative", "twice", "count", "negative count", "page", "width", "cached"])
def test_accept_leaves_a_bad_sequence_as_it_is(q8, what):
    import torch

    rng = np.random.default_rng(4)
    host, cache = new_cache(q8, rng, 2, 8, 2, 16, 64, False)
    table = np.array([[0, 1, -1], [2, 3, -1]], np.int32)
    cached, fresh, counts = [10, 12], [8, 8], [3, 2]
    paths = np.array([[0, 2, 5, 0, 0], [1, 4, 0, 0, 0]], np.int32)
    if what == "order":
        paths[0] = [0, 5, 2, 0, 0]
    elif what == "past":
        paths[0, 2] = 8
    elif what == "negative":
        paths[0, 0] = -1
    elif what == "twice":
        paths[0] = [1, 2, 2, 0, 0]
    elif what == "count":
        counts[0] = 6
    elif what == "negative count":
        counts[0] = -1
    elif what == "page":
        table[0, 0] = 8
    elif what == "width":
        cached[0], counts[0] = 45, 3  # its fresh tokens lie past the table's last page
    else:
        cached[0] = -1
    lens = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    q8.q8_kv_accept(cache, dev(table), dev(cached), dev(fresh), dev(paths), dev(counts), lens)
    with pytest.raises(q8.Q8Error) as e:
        q8.q8_check()
    assert e.value.status == 8
    assert lens.cpu().tolist() == [cached[0], 14]
    for x in host[:2]:
        old = x.copy()
        for j in range(2):
            s, t = 12 + paths[1, j], 12 + j
            x[:, table[1, t // 16], :, t % 16] = old[:, table[1, s // 16], :, s % 16]
    for a, b in zip(host, tensors(cache)):
        assert equal(a, b)
