"""Attention in 64 bits with q and the softmax weights rounded to a number of f16 parts, and the norm-wise limit that the
kernels' two parts are held to.

The error of a call is measured over all its rows: |y - want| in the 2-norm, against the 2-norm of
R = sqrt(sum_j p_j^2 |v_j|^2), the size of an average of independent values.  What two parts and f32 statistics leave of it:
  - q: a value scaled to at most 2 is off by 2^-23 of the row's largest; over a contraction of D independent products, with
    |q|_max of 4.5 times its deviation, that is 2^-23 / sqrt(3) * 4.5 times the scores' deviation of 1.5: 2^-21.1;
  - scores: D/16 <= 8 accumulations, each losing at most 2^-23 of the sum so far, which grows like a random walk (2/3 of
    its end on average): 8 * 2/3 * 2^-23 * 1.5 = 2^-20, twice that for two halves of an instruction's products: 2^-19;
  - weights: the exponent's argument, below 32 and rounded twice (2^-24 * 32 * ln 2, a third of it on average): 2^-21;
    ex2.approx and the two parts: 2^-22 each;
  - products: at most 64 accumulations into O between two sums rounded to nearest, 64 * 2/3 * 2^-23 = 2^-17.6;
  - l and the quotient: 2^-22.
Together below 2^-17: the limit is 2^-16.  One part instead of two is off by 2^-11 / sqrt(3) of each weight or value of q at
most, and by 2^-13 or more on average over the mantissas: eight times the limit."""
import numpy as np

LIMIT = 2.0 ** -16


def parts(x, n):
    """x as the sum of n f16 parts (None: as it is)."""
    if n is None:
        return x
    got, rest = np.zeros_like(x), x
    for _ in range(n):
        got = got + rest.astype(np.float16).astype(np.float64)
        rest = x - got
    return got


def attention(case, masks=None, q_parts=None, p_parts=None, layer=0):
    """(y, R) of every row and head: [total][heads][d] and [total][heads].

    With q_parts a row of q is scaled by a power of two to below 2 and rounded; with p_parts the weights are, as the kernels
    have them: 2^6 at the row's maximum, for int8 times the value's scale over a power of two that no scale exceeds."""
    c = case
    y, size = np.zeros((c.total, c.heads, c.d)), np.zeros((c.total, c.heads))
    group, at = c.heads // c.kv_heads, 0
    for b, (n, f) in enumerate(zip(c.cached, c.fresh)):
        pos = np.arange(n + f)
        pg, off = c.table[b][pos // c.page], pos % c.page
        for h in range(c.kv_heads):
            k, v = c.k[layer][pg, h, off], c.v[layer][pg, h, off]
            vs = None if c.vs is None else c.vs[layer][pg, h, off].astype(np.float64)
            norm = np.linalg.norm(v, axis=1)
            seen = np.ones((f, n + f), bool)
            for i in range(f):
                for j in range(f):
                    seen[i, n + j] = j <= i if masks is None else (int(masks[at + i]) >> j) & 1
            for a in range(h * group, (h + 1) * group):
                x = c.q[at:at + f, a * c.d:(a + 1) * c.d].astype(np.float64)
                if q_parts:
                    two = 2.0 ** np.floor(np.log2(np.abs(x).max(1, keepdims=True)))
                    x = parts(x / two, q_parts) * two
                s = np.where(seen, (x @ k.T) * c.d ** -0.5 * np.log2(np.e), -np.inf)
                p = np.exp2(s - np.maximum(s.max(1, keepdims=True), -1e300))
                total = np.maximum(p.sum(1, keepdims=True), 1e-300)
                if vs is None:
                    o = parts(64 * p, p_parts) / 64 @ v
                else:
                    big = np.where(seen, vs, 0).max(1, keepdims=True)
                    two = 2.0 ** np.ceil(np.log2(np.maximum(big, 1e-300)))
                    o = (parts(64 * p * np.where(seen, vs, 0) / two, p_parts) * two / 64) @ (v / vs[:, None])
                y[at:at + f, a] = o / total
                size[at:at + f, a] = np.sqrt(((p / total) ** 2 * norm ** 2).sum(1))
        at += f
    return y, size


def error(got, want, size):
    """The norm-wise error of y [total][heads * d]."""
    d = np.asarray(got, np.float64).reshape(want.shape) - want
    return float(np.sqrt((d ** 2).sum() / (size ** 2).sum()))
