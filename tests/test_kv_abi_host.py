"""Host-side checks of the key/value cache's entry points: bad arguments are refused before any device work."""
import ctypes

import pytest

import int8_quantized_projection_gb300 as q8p
from int8_quantized_projection_gb300 import _binding, build

FAKE, MISALIGNED = 0x10000, 0x10004  # never dereferenced: every call below fails validation first
P = ctypes.c_void_p
ERR_ARG, ERR_ALIGN = 1, 2
LONG = 1 << 20  # contexts whose attention needs a workspace


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q8p.lib()


def desc(k=FAKE, v=FAKE, ks=None, vs=None, layers=2, n_pages=8, kv_heads=4, page=16, dim=128, dtype=1):
    return _binding.KvCacheDesc(k, v, ks, vs, layers, n_pages, kv_heads, page, dim, dtype)


def ref(d):
    return ctypes.cast(ctypes.pointer(d), P)


BAD_CACHES = [dict(k=None), dict(v=None), dict(layers=0), dict(n_pages=0), dict(kv_heads=0), dict(kv_heads=1025), dict(page=0),
              dict(page=8), dict(page=24), dict(page=-16), dict(dim=96), dict(dim=256), dict(dtype=0), dict(dtype=3),
              dict(ks=FAKE), dict(dtype=2), dict(dtype=2, ks=FAKE), dict(n_pages=1 << 28, page=16),
              dict(n_pages=1 << 26, kv_heads=4, page=16)]


def append(lib, d, layer=0, k=FAKE, v=FAKE, slots=FAKE, tokens=3):
    return lib.q8_kv_append(ref(d) if d is not None else None, layer, P(k), P(v), P(slots), tokens, P(0))


def attend(lib, d, layer=0, q=FAKE, heads=28, table=FAKE, max_pages=4, cached=FAKE, starts=FAKE, batch=2, masks=0, tokens=6,
           max_fresh=3, max_len=64, y=FAKE, qs=0, ds=0, ws=FAKE, nbytes=1 << 30):
    return lib.q8_tree_attention(ref(d) if d is not None else None, layer, P(q), heads, 0.1, P(table), max_pages, P(cached),
                                 P(starts), batch, P(masks), tokens, max_fresh, max_len, P(y), P(qs), P(ds), P(ws), nbytes,
                                 P(0))


def accept(lib, d, table=FAKE, max_pages=4, cached=FAKE, fresh=FAKE, batch=2, paths=FAKE, counts=FAKE, width=8, lens=FAKE):
    return lib.q8_kv_accept(ref(d) if d is not None else None, P(table), max_pages, P(cached), P(fresh), batch, P(paths),
                            P(counts), width, P(lens), P(0))


def plan(lib, cached=FAKE, fresh=FAKE, batch=2, held=0, free=FAKE, n_free=4, table=FAKE, max_pages=4, page=16, n_pages=8,
         parents=0, tokens=6, starts=FAKE, slots=FAKE, positions=FAKE, masks=0, needed=FAKE, held_out=0):
    return lib.q8_kv_plan(P(cached), P(fresh), batch, P(held), P(free), n_free, P(table), max_pages, page, n_pages, P(parents),
                          tokens, P(starts), P(slots), P(positions), P(masks), P(needed), P(held_out), P(0))


@pytest.mark.parametrize("call", [append, attend, accept])
def test_cache_descriptors(lib, call):
    assert call(lib, None) == ERR_ARG
    for bad in BAD_CACHES:
        assert call(lib, desc(**bad)) == ERR_ARG, bad
    for bad in (dict(k=MISALIGNED), dict(v=MISALIGNED), dict(dtype=2, ks=MISALIGNED, vs=FAKE),
                dict(dtype=2, ks=FAKE, vs=MISALIGNED)):
        assert call(lib, desc(**bad)) == ERR_ALIGN, bad


def test_append_arguments(lib):
    for kw in (dict(k=0), dict(v=0), dict(slots=0), dict(tokens=0), dict(tokens=-1), dict(layer=-1), dict(layer=2),
               dict(tokens=1 << 27), dict(tokens=1 << 31)):
        assert append(lib, desc(), **kw) == ERR_ARG, kw
    for kw in (dict(k=MISALIGNED), dict(v=MISALIGNED), dict(slots=MISALIGNED)):
        assert append(lib, desc(), **kw) == ERR_ALIGN, kw


def test_attention_arguments(lib):
    for kw in (dict(q=0), dict(table=0), dict(cached=0), dict(starts=0), dict(y=0), dict(y=0, qs=FAKE), dict(y=0, ds=FAKE),
               dict(qs=FAKE), dict(layer=2), dict(layer=-1), dict(heads=0), dict(heads=30), dict(heads=4 * 65), dict(batch=0),
               dict(batch=4097), dict(tokens=0), dict(max_fresh=0), dict(max_fresh=7), dict(max_len=2), dict(max_len=1 << 31),
               dict(max_pages=0), dict(masks=FAKE, tokens=99, max_fresh=65), dict(ws=0, max_len=LONG),
               dict(nbytes=0, max_len=LONG),
               dict(batch=4096, tokens=1 << 23, max_fresh=1 << 23, max_len=1 << 30)):
        assert attend(lib, desc(), **kw) == ERR_ARG, kw
    need = lib.q8_tree_attention_workspace_bytes(ref(desc()), 28, 3)
    assert need > 0 and attend(lib, desc(), nbytes=need - 1, max_len=LONG) == ERR_ARG
    for name in ("q", "table", "cached", "starts", "masks", "y", "ws"):
        assert attend(lib, desc(), **{name: MISALIGNED}) == ERR_ALIGN, name
    assert attend(lib, desc(), qs=MISALIGNED, ds=FAKE) == ERR_ALIGN
    assert attend(lib, desc(), qs=FAKE, ds=MISALIGNED) == ERR_ALIGN


def test_attention_workspace(lib):
    size = lambda heads, fresh, **kw: lib.q8_tree_attention_workspace_bytes(ref(desc(**kw)), heads, fresh)  # noqa: E731
    assert size(30, 1) == 0 and size(28, 0) == 0 and size(28, 1, dim=80) == 0
    assert 0 < size(28, 1) <= size(28, 2) <= size(28, 64) == size(28, 3325)
    # two pieces a CTA of 8 rows: numerators, (m, l) and descriptors
    assert size(28, 1) == 2 * 152 * 8 * 128 * 4 + 2 * 152 * 8 * 8 + 2 * 152 * 16
    assert size(28, 1, dim=64) < size(28, 1)


def test_attention_needs_a_workspace(lib):
    needs = lambda heads, batch, fresh, most, **kw: lib.q8_tree_attention_needs_workspace(  # noqa: E731
        ref(desc(**kw)), heads, batch, fresh, most)
    for heads, fresh in ((28, 1), (28, 2), (28, 16)):  # 8, 16 and 128 rows a unit
        assert needs(heads, 2, fresh, 300) == 0 and needs(heads, 2, fresh, LONG) == 1
        assert needs(heads, 38, fresh, 300) == 0
    assert needs(28, 1, 1, 4098) == 0 and needs(28, 1, 3325, 3325) == 1
    assert needs(30, 2, 1, 300) == 1 and needs(28, 0, 1, 300) == 1 and needs(28, 2, 0, 300) == 1  # nothing a call would take


def test_accept_arguments(lib):
    for kw in (dict(table=0), dict(cached=0), dict(fresh=0), dict(paths=0), dict(counts=0), dict(lens=0), dict(batch=0),
               dict(batch=4097), dict(width=0), dict(width=65), dict(max_pages=0)):
        assert accept(lib, desc(), **kw) == ERR_ARG, kw
    for name in ("table", "cached", "fresh", "paths", "counts", "lens"):
        assert accept(lib, desc(), **{name: MISALIGNED}) == ERR_ALIGN, name
    assert accept(lib, desc(layers=65536)) == ERR_ARG


def test_plan_arguments(lib):
    for kw in (dict(cached=0), dict(fresh=0), dict(table=0), dict(starts=0), dict(slots=0), dict(positions=0), dict(needed=0),
               dict(parents=FAKE), dict(masks=FAKE), dict(n_free=-1), dict(free=0), dict(batch=0), dict(batch=4097),
               dict(tokens=0), dict(tokens=1 << 31), dict(max_pages=0), dict(page=0), dict(page=20), dict(n_pages=0),
               dict(n_pages=1 << 27)):
        assert plan(lib, **kw) == ERR_ARG, kw
    for name in ("cached", "fresh", "held", "free", "table", "starts", "slots", "positions", "needed", "held_out"):
        assert plan(lib, **{name: MISALIGNED}) == ERR_ALIGN, name
    assert plan(lib, parents=MISALIGNED, masks=FAKE) == ERR_ALIGN


def test_status_has_a_text(lib):
    assert b"out of range" in lib.q8_strerror(8)


def test_binding_refuses_tensors_it_cannot_pass_on():
    import torch

    k = torch.zeros(1, 2, 1, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        q8p.KvCache(k, k)  # not on the GPU
    with pytest.raises(ValueError):
        q8p.KvCache(k[0], k[0])
    with pytest.raises(ValueError):
        q8p.KvCache(k, k[..., :32])
    with pytest.raises(ValueError):
        q8p.KvCache(k.float(), k.float())
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        q8p.q8_kv_plan(i, i, i, i.view(4, 1), 16, 8, i, i, i, i)
