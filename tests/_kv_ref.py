"""Plain references of the paged key/value cache's calls (numpy, 64 bits, loops over the definition) and the
limits their f32 results are held to."""
import numpy as np


def pages_of(tokens, page):
    return -(-tokens // page)


def plan(cached, fresh, page, free, table, tokens, parents=None, held=None):
    """What q8_kv_plan writes: (table, starts, slots, positions, masks, needed, held_out)."""
    table = table.copy()
    starts, at, used = [0], 0, 0
    slots = np.full(tokens, -1, np.int64)
    positions, masks, held_out = {}, {}, []
    for b, (c, f) in enumerate(zip(cached, fresh)):
        have = pages_of(c, page) if held is None else held[b]
        want = pages_of(c + f, page)
        for i in range(have, want):
            if used < len(free):
                table[b, i] = free[used]
            used += 1
        held_out.append(max(have, want))
        opened = used - max(0, want - have)
        for i in range(f):
            pos = c + i
            pi = pos // page
            got = pi < have or opened + (pi - have) < len(free)
            slots[at + i] = table[b, pi] * page + pos % page if got else -1
            positions[at + i] = pos
            if parents is not None:
                p = parents[at + i]
                masks[at + i] = (1 << i) | (masks[at + p] if p >= 0 else 0)
                positions[at + i] = c + bin(masks[at + i]).count("1") - 1
        at += f
        starts.append(at)
    return table, starts, slots, positions, masks, used, held_out


def attention(q, k, v, page, table, cached, fresh, heads, scale, masks=None):
    """y [total][heads * d] in 64 bits and, beside each value, the limit an f32 result is held to.

    k, v: float64 [n_pages][kv_heads][page][d] (the values the cache stands for).

    The limit.  q enters as two f16 parts of its row scaled to [1, 2): each value is off by at most 2^-22 of the
    row's largest.  The tensor core adds D/16 groups of 16 products per part in f32, each group aligned to its
    largest term with 24 bits kept: at most 2 * (D/16) * 17 * 2^-24 < 2^-15 of sum |q||k| for D = 128 in the worst
    case, of which truncations of alternating terms reach a small part; the bound used is 2^-18 of the row's
    B = scale * max_j (max|q| * sum|k_j|), which is itself several times sum |q||k|.  An error d of the exponent
    changes every weight by a factor within 1 +- d, so y by at most 2 d * sum p|v|.  ex2.approx (2^-22), the split
    of the weights (2^-22), the scales' products (2^-24 each) and the quotient (2^-23) stay under 2^-19; the
    sums over n keys add at most (n / 16) * 2^-22 in the MMA and in l together."""
    d = k.shape[-1]
    kv_heads = k.shape[1]
    group = heads // kv_heads
    total = int(sum(fresh))
    y = np.zeros((total, heads, d))
    lim = np.zeros((total, heads, d))
    at = 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        n = c + f
        pos = np.arange(n)
        pg, off = table[b][pos // page], pos % page
        for i in range(f):
            seen = pos < c
            for j in range(f):
                see = j <= i if masks is None else (int(masks[at + i]) >> j) & 1
                seen[c + j] = bool(see)
            if not seen.any():
                continue
            for h in range(heads):
                kh = k[pg[seen], h // group, off[seen]]
                vh = v[pg[seen], h // group, off[seen]]
                x = q[at + i, h * d:(h + 1) * d].astype(np.float64)
                s = kh @ x * scale
                e = np.exp(s - s.max())
                e /= e.sum()
                y[at + i, h] = e @ vh
                big = scale * np.abs(x).max() * np.abs(kh).sum(-1).max()
                rel = 2 * big * 2.0 ** -18 + 2.0 ** -19 + len(e) * 2.0 ** -26
                lim[at + i, h] = rel * (e @ np.abs(vh)) + 2.0 ** -100
        at += f
    return y.reshape(total, heads * d), lim.reshape(total, heads * d)


def tree(rng, n, reach=8):
    """Parents of a random draft tree of n nodes and its masks."""
    parents, masks = [], []
    for i in range(n):
        p = int(rng.integers(max(-1, i - reach), i))
        parents.append(p)
        masks.append((1 << i) | (masks[p] if p >= 0 else 0))
    return parents, masks


def as_i64(masks):
    return np.array([m - (1 << 64) if m >> 63 else m for m in masks], np.int64)


class Case:
    """A filled cache with a shuffled page table: arrays on the host, tensors on the device."""

    def __init__(self, seed, cached, fresh, heads, kv_heads, d, page, int8, layers=1, spare=3, junk=0.0):
        import torch

        import int8_quantized_projection_gb300 as q8

        rng = np.random.default_rng(seed)
        self.rng, self.page, self.heads, self.kv_heads, self.d = rng, page, heads, kv_heads, d
        self.cached, self.fresh = list(cached), list(fresh)
        need = [pages_of(c + f, page) for c, f in zip(cached, fresh)]
        n_pages = sum(need) + spare
        ids = rng.permutation(n_pages)
        width = max(max(need), 1) + 1
        self.table = np.full((len(need), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (layers, n_pages, kv_heads, page, d)
        if int8:
            self.kc, self.vc = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
            self.ks, self.vs = (rng.uniform(0.005, 0.03, shape[:-1]).astype(np.float32) for _ in range(2))
            self.k = self.kc.astype(np.float64) * self.ks[..., None]
            self.v = self.vc.astype(np.float64) * self.vs[..., None]
        else:
            self.kc, self.vc = (rng.normal(0, 1, shape).astype(np.float16) for _ in range(2))
            self.ks = self.vs = None
            self.k, self.v = self.kc.astype(np.float64), self.vc.astype(np.float64)
        total = int(sum(fresh))
        self.total = total
        self.q = (rng.normal(0, 1.5, (total, heads * d))).astype(np.float32)
        self.starts = np.concatenate([[0], np.cumsum(fresh)]).astype(np.int32)
        self.layers = layers
        self.torch, self.q8 = torch, q8

    def dev(self, a):
        return None if a is None else self.torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def cache(self):
        return self.q8.KvCache(self.dev(self.kc), self.dev(self.vc), self.dev(self.ks), self.dev(self.vs))

    def reference(self, masks=None, scale=None, layer=0):
        return attention(self.q, self.k[layer], self.v[layer], self.page, self.table, self.cached, self.fresh, self.heads,
                         self.d ** -0.5 if scale is None else scale, masks)

    def run(self, masks=None, plane=False, layer=0, tokens=None, **kw):
        """y (and plane) of the fresh rows; `tokens` > total pads the rows."""
        t = self.torch
        rows = tokens or self.total
        q = np.full((rows, self.heads * self.d), np.nan, np.float32)
        q[:self.total] = self.q
        y = t.full((rows, self.heads * self.d), float("nan"), device="cuda")
        qs = t.full((rows, self.heads * self.d), 77, dtype=t.int8, device="cuda") if plane else None
        ds = t.full((rows, self.heads * self.d // 32), 77, dtype=t.int32, device="cuda") if plane else None
        m = None
        if masks is not None:
            m = np.zeros(rows, np.int64)
            m[:self.total] = as_i64(masks)
        kw.setdefault("max_fresh", max(self.fresh))
        kw.setdefault("max_len", max(c + f for c, f in zip(self.cached, self.fresh)))
        self.q8.q8_tree_attention(self.cache(), layer, self.dev(q), self.dev(self.table),
                                  self.dev(np.array(self.cached, np.int32)), self.dev(self.starts), y, qs=qs, ds=ds,
                                  masks=self.dev(m), **kw)
        return (y, qs, ds) if plane else y


def assert_within(got, want, lim, what=""):
    got = np.asarray(got, np.float64)
    assert not np.isnan(got).any(), f"{what}: {int(np.isnan(got).sum())} unwritten (NaN) values"
    err = np.abs(got - want)
    worst = float((err / np.maximum(lim, 1e-300)).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: error is {worst:.3g} times the limit (largest {err.max():.3g})"
    return worst
