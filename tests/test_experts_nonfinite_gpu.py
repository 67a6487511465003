"""Gate and up on planes and weights whose scales are infinite or NaN: the plane is the encoding that swiglu_quant gives the two
products, in the stream and in the tiles, and the other rows stay as they are."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu

INF, NAN = 0x7C00, 0x7E00  # f16


@pytest.mark.parametrize("tokens", [9, 300], ids=["stream", "tiles"])
@pytest.mark.parametrize("k", [512, 288])
def test_gate_up(q8, tokens, k):
    import torch

    experts, nf = 2, 96
    g = np.random.default_rng([tokens, k])
    (bg, _), (bu, _) = (ref.weights_of(g, experts, nf, k) for _ in range(2))
    offsets, rows = ref.groups(g, experts, tokens, 1, "spread")
    qs, ds, _ = ref.plane_of(g, tokens, k)
    dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    do, dr = dev(offsets, np.int32), dev(rows, np.int32)

    def planes(ds, bg, bu):
        """The call's plane, and swiglu_quant's of the two products."""
        dg, du, dq, dd = dev(bg), dev(bu), dev(qs), dev(ds)
        mine, want = q8.empty_plane(tokens, nf), q8.empty_plane(tokens, nf)
        q8.q8_0_experts_gate_up(dg, du, experts, nf, k, dq, dd, do, *mine, rows=dr, top_k=1)
        y = [torch.empty(tokens, nf, device="cuda") for _ in range(2)]
        for w, o in zip((dg, du), y):
            q8.q8_0_experts_gemm(w, experts, nf, k, dq, dd, do, o, rows=dr, top_k=1)
        q8.swiglu_quant(*y, None, *want)
        q8.q8_check()
        return [t.cpu().numpy() for t in (*mine, *want)], [t.cpu().numpy() for t in y]

    (q0, d0, wq, wd), _ = planes(ds, bg, bu)
    assert np.array_equal(q0, wq) and np.array_equal(d0, wd)  # finite: the same bits as well
    source = rows
    for word in (INF, NAN):
        # an activation's first block, and a whole row of them; a code of 0 there, so that an infinite scale gives NaN as well
        bad, codes = ds.copy(), qs.copy()
        one, all_ = int(source[1]), int(source[tokens - 2])
        bad[one, 0] = (bad[one, 0] & ~0xffff) | word
        bad[all_] = (bad[all_] & ~0xffff) | word
        qs[all_] = 0
        (q1, d1, wq, wd), y = planes(bad, bg, bu)
        assert np.isnan(y[0][tokens - 2]).all() and not np.isfinite(y[0][1]).any()
        assert np.array_equal(q1, wq) and np.array_equal(d1, wd)
        halves = (d1[tokens - 2].view(np.uint32) & 0xffff).astype(np.uint16).view(np.float16)
        assert np.isnan(halves).all() and not q1[tokens - 2].any()  # seen as NaN, not as zeros
        keep = ~np.isin(np.arange(tokens), [1, tokens - 2])
        assert np.array_equal(q1[keep], q0[keep]) and np.array_equal(d1[keep], d0[keep])
        qs[:] = codes
        # one weight row of gate, one of up: a value of each block they lie in
        for which in range(2):
            blobs = [bg.copy(), bu.copy()]
            blobs[which].reshape(experts * nf, k // 32, 34)[40, 1, :2] = np.frombuffer(np.uint16(word).tobytes(), np.uint8)
            (q2, d2, wq, wd), _ = planes(ds, *blobs)
            assert np.array_equal(q2, wq) and np.array_equal(d2, wd)
            first = slice(0, int(offsets[1]))
            assert np.array_equal(q2[first, 64:], q0[first, 64:]) and np.array_equal(q2[first, :32], q0[first, :32])
            assert np.array_equal(q2[int(offsets[1]):], q0[int(offsets[1]):])
