"""The tiles with as many sorted rows as a call takes: the numbers of the rows plus a step pass 31 bits."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu


def test_most_rows(q8):
    import torch

    pairs, plane_rows, k, step = 2 ** 31 - 257, 7, 32, 7 << 25
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 190 << 30:
        pytest.skip("needs 168 GB: 64 bytes of activations a row beside the scales, the rows and the results")
    g = np.random.default_rng(0)
    blob, w = ref.weights_of(g, 1, 1, k)
    qs, ds, x = ref.plane_of(g, plane_rows, k)
    dw, dq, dd = (torch.from_numpy(a).cuda() for a in (blob, qs, ds))
    rows = torch.empty(pairs, dtype=torch.int32, device="cuda")
    for r in range(0, pairs, step):
        rows[r:r + step] = torch.arange(min(step, pairs - r), dtype=torch.int32, device="cuda") % plane_rows
    offsets = torch.tensor([0, pairs], dtype=torch.int32, device="cuda")
    y = torch.full((pairs, 1), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(dw, 1, 1, k, dq, dd, offsets, y, rows=rows, top_k=1)
    q8.q8_check()
    want, lim = ref.product(w, x, np.array([0, plane_rows]), np.arange(plane_rows))
    first = y[:plane_rows, 0].clone()
    assert np.all(np.abs(first.cpu().numpy() - want[:, 0]) <= lim[:, 0])
    for r in range(0, pairs, step):
        n = min(step, pairs - r)
        assert torch.equal(y[r:r + n, 0], first.repeat(-(-n // plane_rows))[:n])
    del y, rows
    torch.cuda.empty_cache()
