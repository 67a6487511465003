"""rmsnorm_residual_quant against its definition in 64 bits."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu


def inputs(g, rows, d, top_k, dense, post, gate, holes=True):
    f = lambda *s: g.standard_normal(s).astype(np.float32)  # noqa: E731
    a = dict(x=f(rows, d) * 3, b=f(rows, d) if dense else None, w_post=1 + 0.2 * f(d) if post else None,
             gate={"none": None, "channel": f(1, d), "row": f(rows, d)}[gate], w=1 + 0.2 * f(d), ye=None, places=None, weights=None)
    if top_k:
        count = rows * top_k + 3
        a["ye"] = f(count, d)
        a["places"] = g.permutation(count)[:rows * top_k].reshape(rows, top_k).astype(np.int32)
        if holes:
            a["places"][g.random((rows, top_k)) < 0.2] = -1
        a["weights"] = g.random((rows, top_k)).astype(np.float32)
    return a


def call(q8, a, alpha=0.75, eps_post=1e-5, eps=1e-6, plane=True, y=True, h=True, pad=0, in_place=False):
    import torch

    t = {k: torch.from_numpy(v).cuda() if v is not None else None for k, v in a.items()}
    rows, d = t["x"].shape
    nan = lambda: torch.full((rows, d), float("nan"), device="cuda")  # noqa: E731
    ho = t["x"] if in_place else nan() if h else None
    yo = nan() if y else None
    qs, ds = q8.empty_plane(max(1, rows + pad), d) if plane else (None, None)
    if plane:
        qs.fill_(3), ds.fill_(3)
    q8.rmsnorm_residual_quant(t["x"], ho, b=t["b"], expert_rows=t["ye"], places=t["places"], weights=t["weights"],
                              w_post=t["w_post"], eps_post=eps_post, gate=t["gate"], residual_scale=alpha,
                              w=t["w"] if plane or y else None, eps=eps, y=yo, qs=qs, ds=ds)
    q8.q8_check()
    return [None if v is None else v.cpu().numpy() for v in (ho, yo, qs, ds)]


def check(a, got, alpha=0.75, eps_post=1e-5, eps=1e-6):
    h, hl, y, yl = ref.residual_norm(a["x"], alpha, a["b"], a["ye"], a["places"], a["weights"], a["w_post"], eps_post, a["gate"],
                                     a["w"], eps)
    gh, gy, qs, ds = got
    if gh is not None:
        assert np.all(np.abs(gh - h) <= hl + 1e-38)
    if gy is not None:
        assert np.all(np.abs(gy - y) <= yl + 1e-38)
    if qs is not None:
        ref.check_plane(qs, ds, y, yl)
        assert not qs[len(h):].any() and not ds[len(h):].any()


@pytest.mark.parametrize("rows,d", [(1, 32), (3, 64), (1, 3584), (5, 4096), (2, 4128), (7, 8192), (1, 32768), (300, 96), (161, 3584),
                                    (400, 1440), (200, 8224)])
@pytest.mark.parametrize("top_k,dense,post,gate", [(0, True, False, "none"), (0, True, True, "channel"), (1, False, True, "none"),
                                                   (8, False, False, "row"), (3, True, True, "row"), (16, True, True, "channel")])
def test_norm(q8, rows, d, top_k, dense, post, gate):
    if rows * d * max(top_k, 1) > 5_000_000:
        rows = max(1, 5_000_000 // (d * top_k))
    a = inputs(np.random.default_rng([rows, d, top_k]), rows, d, top_k, dense, post, gate)
    check(a, call(q8, a, pad=rows % 3))


@pytest.mark.parametrize("rows,d", [(1, 3584), (250, 512), (170, 5120)])
def test_outputs_chosen(q8, rows, d):
    a = inputs(np.random.default_rng(1), rows, d, 4, True, True, "channel")
    whole = call(q8, a)
    check(a, whole)
    for kw in (dict(y=False), dict(plane=False), dict(h=False), dict(h=False, y=False), dict(plane=False, h=False),
               dict(plane=False, y=False), dict(in_place=True)):
        got = call(q8, a, **kw)
        for one, other in zip(got, whole):  # the same bits whichever outputs are written
            assert one is None or np.array_equal(one, other), kw
        if kw.get("in_place"):
            assert got[0] is not None


def test_no_rows(q8):
    a = inputs(np.random.default_rng(1), 0, 64, 0, True, True, "none")
    got = call(q8, a, pad=5)
    assert not got[2].any() and not got[3].any()
    call(q8, a, plane=False)


def test_zero_rows_and_holes(q8):
    a = inputs(np.random.default_rng(2), 6, 128, 2, False, True, "none")
    a["places"][:3] = -1  # no expert: b' is 0, so h is the scaled residual
    a["weights"][:3] = np.nan
    a["x"][1] = 0
    got = call(q8, a)
    assert np.array_equal(got[0][:3], np.float32(0.75) * a["x"][:3])
    assert not got[1][1].any() and not got[2][1].any()
    a["weights"][:3] = 0
    check(a, got)


def test_places_out_of_range(q8):
    import torch

    a = inputs(np.random.default_rng(3), 5, 96, 2, True, False, "none", holes=False)
    good = a["places"].copy()
    for bad in (-2, len(a["ye"]), 1 << 30, -(1 << 31)):
        a["places"] = good.copy()
        a["places"][2, 1] = bad
        t = {k: torch.from_numpy(v).cuda() if v is not None else None for k, v in a.items()}
        h = torch.empty_like(t["x"])
        q8.rmsnorm_residual_quant(t["x"], h, b=t["b"], expert_rows=t["ye"], places=t["places"], weights=t["weights"])
        with pytest.raises(q8.Q8Error, match="DATA"):
            q8.q8_check()
        a["places"][2, 1] = -1
        want, lim, _, _ = ref.residual_norm(a["x"], 1.0, a["b"], a["ye"], a["places"], a["weights"])
        assert np.all(np.abs(h.cpu().numpy() - want) <= lim)


def test_nonfinite_rows_stay_apart(q8):
    a = inputs(np.random.default_rng(4), 300, 256, 2, True, True, "channel", holes=False)
    clean = call(q8, a)
    a["x"][7, 3] = np.inf
    a["b"][150, 0] = np.nan
    got = call(q8, a)
    keep = np.ones(300, bool)
    keep[[7, 150]] = False
    assert np.array_equal(got[0][keep], clean[0][keep]) and np.array_equal(got[1][keep], clean[1][keep])
    assert np.isnan(got[0][150]).all() and not np.isfinite(got[1][7]).all()


def test_refusals(q8):
    import torch

    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    for kw in (dict(b=x[:3]), dict(b=x.half()), dict(b=x.cpu()), dict(b=x, w=w[:32], y=y), dict(b=x, gate=x[:2]), dict(b=x, places=x),
               dict(expert_rows=x), dict(expert_rows=x, places=torch.zeros(4, 1, dtype=torch.int32, device="cuda")),
               dict(b=x, w=w, y=y[:3]), dict(b=x, w=w, qs=torch.empty(4, 64, dtype=torch.int8, device="cuda"))):
        with pytest.raises(ValueError):
            q8.rmsnorm_residual_quant(x, h, **kw)
    for kw in (dict(), dict(b=x, y=y), dict(b=x, w=w), dict(b=h), dict(b=x, residual_scale=float("nan"))):
        with pytest.raises(q8.Q8Error, match="ARG"):
            q8.rmsnorm_residual_quant(x, h, **kw)
    q8.rmsnorm_residual_quant(x, h, b=y)
    q8.q8_check()
