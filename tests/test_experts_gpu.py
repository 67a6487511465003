"""q8_0_experts_gemm and q8_0_experts_gate_up against their definition in 64 bits."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu

# experts, n, k, tokens, top_k, kind: one block a row, odd widths, rows of blocks without common alignment, one token, empty
# experts, one expert with everything, pairs without expert, few and many rows
SHAPES = [(1, 1, 32, 1, 1, "spread"), (4, 17, 64, 3, 2, "spread"), (8, 33, 96, 5, 4, "gaps"), (3, 128, 256, 1, 3, "spread"),
          (8, 100, 512, 9, 2, "one"), (16, 48, 2304, 2, 8, "spread"), (5, 130, 1440, 40, 2, "skew"), (64, 65, 768, 30, 6, "gaps"),
          (2, 257, 1024, 70, 1, "skew"), (4, 64, 7456, 6, 2, "spread"), (2, 31, 18944, 5, 1, "spread"),
          (3, 129, 512, 700, 2, "skew"), (6, 200, 288, 400, 2, "gaps"), (4, 384, 2560, 600, 2, "one"), (2, 96, 32, 500, 1, "spread"),
          (160, 40, 256, 300, 8, "spread")]


def make(experts, n, k, tokens, top_k, kind, gather, pads=0, seed=0):
    g = np.random.default_rng([experts, n, k, tokens, top_k, seed])
    blob, w = ref.weights_of(g, experts, n, k)
    offsets, rows = ref.groups(g, experts, tokens, top_k, kind)
    pairs = tokens * top_k
    qs, ds, x = ref.plane_of(g, tokens if gather else pairs, k, (tokens if gather else pairs) + pads)
    source = rows // top_k if gather else np.arange(pairs)
    return blob, w, offsets, rows, qs, ds, x, source


def cuda(*arrays):
    import torch

    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gemm(q8, shape, gather):
    import torch

    experts, n, k, tokens, top_k, kind = shape
    blob, w, offsets, rows, qs, ds, x, source = make(*shape, gather)
    dw, dq, dd, do, dr = cuda(blob, qs, ds, offsets.astype(np.int32), rows.astype(np.int32))
    y = torch.full((tokens * top_k, n), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(dw, experts, n, k, dq, dd, do, y, rows=dr if gather else None, top_k=top_k)
    q8.q8_check()
    want, lim = ref.product(w, x, offsets, source)
    got, total = y.cpu().numpy(), int(offsets[-1])
    assert np.all(np.abs(got[:total] - want) <= lim)
    assert np.isnan(got[total:]).all()  # rows behind the last expert's are left
    again = torch.empty_like(y)
    q8.q8_0_experts_gemm(dw, experts, n, k, dq, dd, do, again, rows=dr if gather else None, top_k=top_k)
    assert torch.equal(again[:total], y[:total])


@pytest.mark.parametrize("shape", [s[:1] + (-(-s[1] // 32) * 32,) + s[2:] for s in SHAPES], ids=str)
def test_gate_up(q8, shape):
    import torch

    experts, nf, k, tokens, top_k, kind = shape
    blob, w, offsets, rows, qs, ds, x, source = make(*shape, True, pads=3)
    blob2, w2 = ref.weights_of(np.random.default_rng(9), experts, nf, k)
    dg, du, dq, dd, do, dr = cuda(blob, blob2, qs, ds, offsets.astype(np.int32), rows.astype(np.int32))
    pairs, total = tokens * top_k, int(offsets[-1])
    qo = torch.full((pairs + 5, nf), 77, dtype=torch.int8, device="cuda")
    so = torch.full((pairs + 5, nf // 32), 77, dtype=torch.int32, device="cuda")
    q8.q8_0_experts_gate_up(dg, du, experts, nf, k, dq, dd, do, qo, so, rows=dr, top_k=top_k)
    q8.q8_check()
    (gt, gl), (ut, ul) = ref.product(w, x, offsets, source), ref.product(w2, x, offsets, source)
    y, lim = ref.swiglu(gt, gl, ut, ul)
    ref.check_plane(qo.cpu().numpy(), so.cpu().numpy(), y, lim)
    assert (qo[total:] == 77).all() and (so[total:] == 77).all()


@pytest.mark.parametrize("tokens", [6, 900])
def test_bad_offsets_and_rows(q8, tokens):
    import torch

    experts, n, k, top_k = 4, 48, 512, 2
    blob, w, offsets, rows, qs, ds, x, source = make(experts, n, k, tokens, top_k, "spread", True)
    dw, dq, dd = cuda(blob, qs, ds)
    want, lim = ref.product(w, x, offsets, source)
    pairs = tokens * top_k

    def run(offsets, rows):
        y = torch.full((pairs, n), float("nan"), device="cuda")
        do, dr = cuda(np.asarray(offsets, np.int32), np.asarray(rows, np.int32))
        q8.q8_0_experts_gemm(dw, experts, n, k, dq, dd, do, y, rows=dr, top_k=top_k)
        with pytest.raises(q8.Q8Error, match="DATA"):
            q8.q8_check()
        q8.q8_check()
        return y.cpu().numpy()

    def same(got, keep):
        assert np.all(np.abs(got[keep] - want[keep]) <= lim[keep]) and np.isnan(got[~keep]).all()

    at = np.arange(pairs)
    bad = rows.copy()
    bad[[0, pairs // 2]] = [-1, tokens * top_k + 5]  # two rows whose pair is out of range
    same(run(offsets, bad), ~np.isin(at, [0, pairs // 2]))
    for far in (1 << 30, -(1 << 30)):
        bad = rows.copy()
        bad[1] = far
        same(run(offsets, bad), at != 1)
    low = offsets.copy()
    low[0] = -4  # the first expert starts before the rows
    same(run(low, rows), at >= offsets[1])
    high = offsets.copy()
    high[4] = pairs + 1  # the last one ends behind them
    same(run(high, rows), at < offsets[3])
    swapped = offsets.copy()
    swapped[2] = offsets[1] - 1  # expert 1 has a negative count; expert 2 also gets expert 1's rows
    got = run(swapped, rows)
    keep = (at < offsets[1] - 1) | (at >= offsets[3])
    assert np.all(np.abs(got[keep] - want[keep]) <= lim[keep])


def test_offsets_that_overlap_without_end(q8):
    """Every second expert claims all rows: more items of the stream's line than 31 bits number.  Nothing is computed."""
    import torch

    experts, n, pairs = 1024, 32768, 25000
    w = torch.zeros(experts * n * 34, dtype=torch.uint8, device="cuda")
    qs, ds = q8.empty_plane(pairs, 32)
    qs.zero_(), ds.zero_()
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = pairs
    y = torch.full((pairs, n), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(w, experts, n, 32, qs, ds, offsets, y)
    with pytest.raises(q8.Q8Error, match="DATA"):
        q8.q8_check()
    assert y.isnan().all()


@pytest.mark.parametrize("k,rows", [(10240, 3), (10272, 3), (10240, 40), (10272, 40)])
def test_weights_past_32_bits(q8, k, rows):
    """The last of 96 experts starts 5.3 GB into the blocks and is the only one with rows (with 40 an expert on average: tiles)."""
    import torch

    experts, n, pairs = 96, 5120, 96 * rows
    blob, w = ref.weights_of(np.random.default_rng(3), 1, n, k)
    wd = torch.zeros(experts * n * (k // 32) * 34, dtype=torch.uint8, device="cuda")
    wd[-blob.size:] = torch.from_numpy(blob).cuda()
    qs, ds, x = ref.plane_of(np.random.default_rng(4), 5, k)
    source = np.arange(9) % 5
    rows_ = np.full(pairs, -1, np.int64)
    rows_[:9] = source
    offsets = np.zeros(experts + 1, np.int64)
    offsets[-1] = 9
    dq, dd, do, dr = cuda(qs, ds, offsets.astype(np.int32), rows_.astype(np.int32))
    y = torch.full((pairs, n), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(wd, experts, n, k, dq, dd, do, y, rows=dr, top_k=1)
    q8.q8_check()
    want, lim = ref.product(w, x, np.array([0, 9]), source)
    assert np.all(np.abs(y[:9].cpu().numpy() - want) <= lim) and y[9:].isnan().all()


@pytest.mark.parametrize("k", [256, 288])
@pytest.mark.parametrize("counts", [[0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 0, 112, 113, 127, 128, 129, 143, 145, 255, 256, 257, 0],
                                    [25], [24], [0, 0, 0, 100], [385, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0]])
def test_rows_at_the_edges_of_tiles(q8, counts, k):
    """Every number of rows at which a tile, a step of 16 columns or a copy of 64 rows ends."""
    import torch

    g = np.random.default_rng(len(counts))
    experts, n, nf = len(counts), 160, 96
    offsets = np.concatenate([[0], np.cumsum(counts)])
    total = int(offsets[-1])
    pairs = total + 3
    source = g.integers(0, 50, total)
    rows = np.concatenate([source, [-1, -1, -1]])
    qs, ds, x = ref.plane_of(g, 50, k)
    (blob, w), (bg, wg), (bu, wu) = ref.weights_of(g, experts, n, k), ref.weights_of(g, experts, nf, k), ref.weights_of(g, experts, nf, k)
    dw, dg, du, dq, dd, do, dr = cuda(blob, bg, bu, qs, ds, offsets.astype(np.int32), rows.astype(np.int32))
    y = torch.full((pairs, n), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(dw, experts, n, k, dq, dd, do, y, rows=dr, top_k=1)
    qo = torch.full((pairs, nf), 77, dtype=torch.int8, device="cuda")
    so = torch.full((pairs, nf // 32), 77, dtype=torch.int32, device="cuda")
    q8.q8_0_experts_gate_up(dg, du, experts, nf, k, dq, dd, do, qo, so, rows=dr, top_k=1)
    q8.q8_check()
    want, lim = ref.product(w, x, offsets, source)
    got = y.cpu().numpy()
    assert np.all(np.abs(got[:total] - want) <= lim) and np.isnan(got[total:]).all()
    v, vlim = ref.swiglu(*ref.product(wg, x, offsets, source), *ref.product(wu, x, offsets, source))
    ref.check_plane(qo.cpu().numpy(), so.cpu().numpy(), v, vlim)
    assert (qo[total:] == 77).all() and (so[total:] == 77).all()


def test_no_pairs_at_all(q8):
    import torch

    experts, n, k = 4, 32, 256
    blob, _, _, _, qs, ds, _, _ = make(experts, n, k, 4, 2, "spread", True)
    dw, dq, dd = cuda(blob, qs, ds)
    do, dr = torch.zeros(experts + 1, dtype=torch.int32, device="cuda"), torch.full((8,), -1, dtype=torch.int32, device="cuda")
    y = torch.full((8, n), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(dw, experts, n, k, dq, dd, do, y, rows=dr, top_k=2)
    qo, so = q8.empty_plane(8, n)
    qo.fill_(5)
    q8.q8_0_experts_gate_up(dw, dw, experts, n, k, dq, dd, do, qo, so, rows=dr, top_k=2)
    q8.q8_check()
    assert torch.isnan(y).all() and (qo == 5).all()


@pytest.mark.parametrize("tokens", [5, 600])
def test_extreme_scales(q8, tokens):
    """f16 scales that are subnormal, zero, the largest, infinite: what they multiply follows f32's rules."""
    import torch

    experts, n, k = 2, 40, 512
    blob, w, offsets, rows, qs, ds, x, source = make(experts, n, k, tokens, 1, "spread", True)
    b = blob.reshape(experts * n, k // 32, 34)
    b[0, :, :2] = np.frombuffer(np.float16(6e-8).tobytes(), np.uint8)
    b[1, 3, :2] = np.frombuffer(np.float16(65504).tobytes(), np.uint8)
    b[2, :, :2] = 0
    b[3, 5, :2] = np.frombuffer(np.float16(np.inf).tobytes(), np.uint8)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    q = np.ascontiguousarray(b[..., 2:]).view(np.int8).astype(np.float64)
    dw, dq, dd, do, dr = cuda(b.reshape(-1), qs, ds, offsets.astype(np.int32), rows.astype(np.int32))
    y = torch.empty(tokens, n, device="cuda")
    q8.q8_0_experts_gemm(dw, experts, n, k, dq, dd, do, y, rows=dr, top_k=1)
    q8.q8_check()
    d[3, 5] = 0
    want, lim = ref.product((q * d).reshape(experts, n, k // 32, 32), x, offsets, source)
    got = y.cpu().numpy()
    first = slice(0, int(offsets[1]))  # expert 0 holds the odd rows of blocks
    blocks = (x[source[first], 5] * q[3, 5]).sum(-1)
    assert np.array_equal(got[first, 3][blocks != 0], np.where(blocks > 0, np.inf, -np.inf)[blocks != 0])
    lim[first, 3] = np.inf
    got[first, 3] = want[first, 3]
    assert np.all(np.abs(got - want) <= lim)


def test_refusals(q8):
    import torch

    blob, _, offsets, rows, qs, ds, _, _ = make(4, 32, 256, 6, 2, "spread", True)
    dw, dq, dd, do, dr = cuda(blob, qs, ds, offsets.astype(np.int32), rows.astype(np.int32))
    y = torch.empty(12, 32, device="cuda")
    ok = dict(w=dw, experts=4, n=32, k=256, qs=dq, ds=dd, offsets=do, y=y, rows=dr, top_k=2)
    q8.q8_0_experts_gemm(**ok)
    for kw in (dict(experts=5), dict(n=31), dict(k=288), dict(w=dw[34:]), dict(qs=dq[:, ::2]), dict(ds=dd[:5]), dict(ds=dd.float()),
               dict(offsets=do[:4]), dict(rows=dr[:11]), dict(rows=dr.long()), dict(y=y.half()), dict(y=y[:, :31]), dict(w=dw.cpu())):
        with pytest.raises(ValueError):
            q8.q8_0_experts_gemm(**{**ok, **kw})
    with pytest.raises(q8.Q8Error, match="ARG"):
        q8.q8_0_experts_gemm(**{**ok, "top_k": 0})
    qo, so = q8.empty_plane(12, 32)
    q8.q8_0_experts_gate_up(dw, dw, 4, 32, 256, dq, dd, do, qo, so, rows=dr, top_k=2)
    with pytest.raises(ValueError):
        q8.q8_0_experts_gate_up(dw, dw, 4, 32, 256, dq, dd, do, qo[:11], so[:11], rows=dr, top_k=2)
    with pytest.raises(ValueError):
        q8.q8_0_experts_gate_up(dw, dw[:-34], 4, 32, 256, dq, dd, do, qo, so, rows=dr, top_k=2)
    q8.q8_check()
