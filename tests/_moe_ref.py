"""Plain references of the mixture-of-experts calls (numpy, 64 bits) and the limits their f32 results are held to."""
import numpy as np

from int8_quantized_projection_gb300 import synthetic as syn

U = 2.0 ** -24  # half a step of f32, relative


def route(logits, top_k, mode, scale=1.0, valid=None):
    """What q8_moe_route writes: (ids, weights in 64 bits, offsets, rows, places)."""
    tokens, experts = logits.shape
    ids = np.full((tokens, top_k), -1, np.int64)
    weights = np.zeros((tokens, top_k))
    for t in range(tokens if valid is None else valid):
        fine = [e for e in range(experts) if logits[t, e] > -np.inf]  # false for NaN
        best = sorted(fine, key=lambda e: (-logits[t, e], e))[:top_k]
        if not best:
            continue
        top = float(logits[t, best[0]])
        share = lambda e: 1.0 if logits[t, e] == top else np.exp(float(logits[t, e]) - top)  # noqa: E731
        total = sum(share(e) for e in (best if mode == 1 else fine))
        ids[t, :len(best)] = best
        weights[t, :len(best)] = [scale * share(e) / total for e in best]
    flat = ids.reshape(-1)
    rows = np.full(tokens * top_k, -1, np.int64)
    places = np.full(tokens * top_k, -1, np.int64)
    offsets, at = [0], 0
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        rows[at:at + len(mine)] = mine
        places[mine] = np.arange(at, at + len(mine))
        at += len(mine)
        offsets.append(at)
    return ids, weights, np.array(offsets), rows, places.reshape(tokens, top_k)


def weights_of(g, experts, n, k):
    """(blob uint8 [experts * n * k/32 * 34], values [experts][n][k/32][32] in 64 bits)."""
    blob, d16, q = syn.q8_0_weights(g, experts * n, k)
    d = d16.view(np.float16).astype(np.float64)
    return blob, (q.reshape(experts, n, k // 32, 32) * d.reshape(experts, n, k // 32, 1))


def plane_of(g, rows, k, rows_pad=None):
    """A plane of random codes: (qs, ds int32, values [rows_pad][k/32][32] in 64 bits)."""
    rows_pad = rows if rows_pad is None else rows_pad
    q = np.zeros((rows_pad, k), np.int8)
    q[:rows] = g.integers(-127, 128, size=(rows, k))
    d16 = np.zeros((rows_pad, k // 32), np.uint16)
    d16[:rows] = g.uniform(0.001, 0.05, size=(rows, k // 32)).astype(np.float16).view(np.uint16)
    ssum = q.reshape(rows_pad, -1, 32).astype(np.int64).sum(-1)
    ds = (d16.astype(np.int64) | ((ssum & 0xffff) << 16)).astype(np.uint32).view(np.int32)
    return q, ds, q.reshape(rows_pad, -1, 32) * d16.view(np.float16).astype(np.float64)[:, :, None]


def groups(g, experts, tokens, top_k, kind="spread"):
    """(offsets, rows) of some routing: ``spread``, ``one`` (all on one expert), ``skew`` or ``gaps`` (pairs without expert)."""
    ids = np.full((tokens, top_k), -1, np.int64)
    for t in range(tokens):
        if kind == "one":
            ids[t] = [(experts // 2 + j) % experts for j in range(top_k)]
        else:
            p = np.arange(1, experts + 1.0) ** (-2.0 if kind == "skew" else 0.0)
            ids[t] = g.choice(experts, top_k, replace=False, p=p / p.sum())
    if kind == "gaps":
        ids[g.random((tokens, top_k)) < 0.4] = -1
    flat = ids.reshape(-1)
    order = np.concatenate([np.flatnonzero(flat == e) for e in range(experts)]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])])
    rows = np.full(flat.size, -1, np.int64)
    rows[:order.size] = order
    return offsets, rows


def product(w, x, offsets, source):
    """(y, limit) of the sorted rows: y = sum over blocks.  A block's integer dot product is exact, and so is the product of
    two f16 scales in f32; adding nb terms in any order rounds each partial sum once: at most nb + 8 times 2^-24 of the
    sum of their magnitudes (8: partial sums joined).  Below 2^-126 a scale product loses bits: 2^-149 times 32 * 127^2."""
    experts, n, nb, _ = w.shape
    total = int(offsets[-1])
    y, lim = np.zeros((total, n)), np.zeros((total, n))
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            t = np.einsum("rbj,ibj->rib", x[source[lo:hi]], w[e], optimize=True)
            y[lo:hi], lim[lo:hi] = t.sum(-1), np.abs(t).sum(-1)
    return y, lim * (nb + 8) * U + nb * 2.0 ** -130


def swiglu(g, dg, u, du):
    """(y, limit) of silu(g) * u for g, u off by at most dg, du.  |silu'| < 1.1; the fast exponential is off by at most
    2 + 1.173 |g| steps of 2^-23 and the quotient by 2: under 2^-16 of y for |g| < 88, where silu(g) is g or below 1e-36."""
    s = g / (1 + np.exp(-np.maximum(g, -700)))
    return s * u, 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -16 * np.abs(s * u) + 1e-35


def check_plane(qs, ds, y, lim):
    """The plane's rows encode values within lim of y: each code is the nearest of a scale amax / 127 stored as f16."""
    rows, k = y.shape
    q = qs[:rows].reshape(rows, k // 32, 32).astype(np.float64)
    word = ds[:rows].view(np.uint32)
    d = (word & 0xffff).astype(np.uint16).view(np.float16).astype(np.float64)
    ssum = (word >> 16).astype(np.uint16).view(np.int16)
    assert np.array_equal(ssum, q.sum(-1).astype(np.int64)), "block sums"
    yb, lb = y.reshape(rows, k // 32, 32), lim.reshape(rows, k // 32, 32)
    amax, most = np.abs(yb).max(-1), lb.max(-1)
    step = amax / 127
    half = 2.0 ** -11 * step + 2.0 ** -25  # the scale's rounding to f16, normal or subnormal
    assert np.all(np.abs(d - step) <= half + most / 127 * 1.01 + 2.0 ** -22 * step), "block scales"
    off = np.abs(q * d[..., None] - yb)
    assert np.all(off <= (0.5 * (step + most / 127) * (1 + 2.0 ** -20) + 127 * half + 2 * most)[..., None] + lb), "codes"


def residual_norm(x, alpha, b=None, ye=None, places=None, weights=None, w_post=None, eps_post=0.0, gate=None, w=None, eps=0.0):
    """(h, its limit, y, its limit) in 64 bits.  Sums of m positive squares in f32: a thread adds up to 64, a warp 5 times, then
    up to 16 warps: under 90 roundings, halved by the root; rsqrt 2 steps; two products: 50 x 2^-24 of the result.  An
    error in the values changes the mean by its share."""
    f = lambda a: None if a is None else np.asarray(a, np.float64)  # noqa: E731
    x, b, ye, weights, w_post, gate, w = map(f, (x, b, ye, weights, w_post, gate, w))
    v = np.zeros_like(x) if b is None else b.copy()
    mag = np.abs(v)
    if ye is not None:
        for t in range(x.shape[0]):
            for j in range(places.shape[1]):
                if places[t, j] >= 0:
                    term = weights[t, j] * ye[places[t, j]]
                    v[t] += term
                    mag[t] += np.abs(term)
    lim = mag * U * (0 if ye is None else places.shape[1])

    def norm(v, lim, w, eps):
        ms = (v * v).mean(-1, keepdims=True)
        r = 1 / np.sqrt(ms + eps)
        rel = (np.abs(v) * lim).mean(-1, keepdims=True) / (ms + eps)
        p = v * r * w
        return p, np.abs(p) * (50 * U + rel) + np.abs(r * w) * lim * (1 + rel) * 1.01

    if w_post is not None:
        v, lim = norm(v, lim, w_post, eps_post)
    if gate is not None:
        v, lim = v * gate, lim * np.abs(gate) + np.abs(v * gate) * U
    h = alpha * x + v
    lim = lim + (np.abs(h) + 2 * np.abs(v)) * U * 1.01
    if w is None:
        return h, lim, None, None
    y, ylim = norm(h, lim, w, eps)
    return h, lim, y, ylim
