"""Sorted rows without a product are left as they were, whichever kernels a call takes: rows whose pair is out of range, rows of
experts whose offsets are out of range, rows before the first expert's."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu

EXPERTS, TOP_K = 8, 2
# call, n, k, tokens: the stream with one slice and with several, the tiles; widths at which a warp has one row or four
FORMS = [("gate_up", 64, 512, 6), ("gate_up", 32, 288, 20), ("gate_up", 1280, 3584, 24), ("gate_up", 96, 512, 900),
         ("gemm", 48, 3584, 24), ("gemm", 1500, 7456, 30), ("gemm", 48, 512, 6), ("gemm", 48, 512, 900)]


class Case:
    def __init__(self, q8, call, n, k, tokens):
        import torch

        self.q8, self.call, self.n, self.k = q8, call, n, k
        g = np.random.default_rng([n, k, tokens])
        self.blobs, self.w = zip(*(ref.weights_of(g, EXPERTS, n, k) for _ in range(2 if call == "gate_up" else 1)))
        self.offsets, self.rows = ref.groups(g, EXPERTS, tokens, TOP_K, "spread")
        self.pairs = tokens * TOP_K
        qs, ds, self.x = ref.plane_of(g, tokens, k)
        self.dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()
        self.dw, self.qs, self.ds = [self.dev(b) for b in self.blobs], self.dev(qs), self.dev(ds)
        self.sizes = (EXPERTS, n, k, tokens, TOP_K, self.pairs)

    def run(self, offsets, rows, keep, error=True, part=slice(0, EXPERTS)):
        """One call on `part` of the experts; the rows of `keep` hold their products, the others what they held."""
        import torch

        q8, experts = self.q8, part.stop - part.start
        do = self.dev(offsets, np.int32)[part.start:part.stop + 1]
        dr = self.dev(rows, np.int32)
        dw = [w.view(EXPERTS, -1)[part].reshape(-1) for w in self.dw]
        sizes = (experts,) + self.sizes[1:]
        need = getattr(q8, f"q8_0_experts_{self.call}_workspace_bytes")(*sizes)
        ws = torch.full((max(need, 16),), 0x41, dtype=torch.uint8, device="cuda")  # as f32: 12.08 each
        kw = dict(rows=dr, top_k=TOP_K, workspace=ws)
        if self.call == "gemm":
            y = torch.full((self.pairs, self.n), float("nan"), device="cuda")
            q8.q8_0_experts_gemm(dw[0], experts, self.n, self.k, self.qs, self.ds, do, y, **kw)
        else:
            qo = torch.full((self.pairs, self.n), 77, dtype=torch.int8, device="cuda")
            so = torch.full((self.pairs, self.n // 32), 77, dtype=torch.int32, device="cuda")
            q8.q8_0_experts_gate_up(dw[0], dw[1], experts, self.n, self.k, self.qs, self.ds, do, qo, so, **kw)
        if error:
            with pytest.raises(q8.Q8Error, match="DATA"):
                q8.q8_check()
        q8.q8_check()
        products = [ref.product(w, self.x, self.offsets, self.rows // TOP_K) for w in self.w]
        if self.call == "gemm":
            (want, lim), got = products[0], y.cpu().numpy()
            assert np.isnan(got[~keep]).all()
            assert np.all(np.abs(got[keep] - want[keep]) <= lim[keep])
        else:
            qn, sn = qo.cpu().numpy(), so.cpu().numpy()
            assert (qn[~keep] == 77).all() and (sn[~keep] == 77).all()
            y, lim = ref.swiglu(*products[0], *products[1])
            ref.check_plane(qn[keep], sn[keep], y[keep], lim[keep])


@pytest.fixture(params=FORMS, ids=lambda f: "-".join(map(str, f)))
def case(q8, request):
    return Case(q8, *request.param)


def test_pairs_out_of_range(case):
    bad = case.rows.copy()
    at = np.unique([0, 1, case.pairs // 2, case.pairs - 1])
    bad[at] = [-1, 1 << 30, case.pairs, -(1 << 31)][:len(at)]
    case.run(case.offsets, bad, ~np.isin(np.arange(case.pairs), at))


def test_offsets_out_of_range(case):
    at, offsets = np.arange(case.pairs), case.offsets
    low = offsets.copy()
    low[0] = -4  # the first expert starts before the rows
    case.run(low, case.rows, at >= offsets[1])
    low[1] = -1  # and the second
    case.run(low, case.rows, at >= offsets[2])
    high = offsets.copy()
    high[EXPERTS] = case.pairs + 1  # the last one ends behind them
    case.run(high, case.rows, at < offsets[EXPERTS - 1])


@pytest.mark.parametrize("part", [slice(4, 8), slice(4, 6), slice(0, 5)], ids=str)
def test_part_of_the_experts(case, part):
    """offsets + e0 with the weights from expert e0 on: the other experts' rows are left, and nothing is reported."""
    at = np.arange(case.pairs)
    rows = case.rows.copy()
    keep = (at >= case.offsets[part.start]) & (at < case.offsets[part.stop])
    rows[~keep] = -1  # nobody's: not read for an address, and no error
    case.run(case.offsets, rows, keep, error=False, part=part)


def test_gate_up_of_offsets_that_overlap_without_end(q8):
    """Every second expert claims all rows: more items of the stream's line than 31 bits number.  Nothing is computed."""
    import torch

    experts, n, pairs = 1024, 32768, 25000
    w = torch.zeros(experts * n * 34, dtype=torch.uint8, device="cuda")
    qs, ds = q8.empty_plane(pairs, 32)
    qs.zero_(), ds.zero_()
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = pairs
    offsets[experts] = pairs
    qo, so = q8.empty_plane(pairs, n)
    qo.fill_(77), so.fill_(77)
    q8.q8_0_experts_gate_up(w, w, experts, n, 32, qs, ds, offsets, qo, so)
    with pytest.raises(q8.Q8Error, match="DATA"):
        q8.q8_check()
    assert (qo == 77).all() and (so == 77).all()
