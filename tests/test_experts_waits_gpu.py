"""The experts' tiles and the norms' ring beside other work on the GPU, where their waits take any time and lanes leave them one by
one: the same bits as on a quiet GPU."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu


def beside_copies(call, outputs):
    """The outputs of calls on one stream while another copies back and forth, and of one call alone."""
    import torch

    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    other, (a, b) = torch.cuda.Stream(), (torch.zeros(1 << 26, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    for _ in range(12):
        with torch.cuda.stream(other):
            for _ in range(6):
                a.copy_(b), b.copy_(a)
        for t in outputs:
            t.zero_()
        call()
        torch.cuda.current_stream().synchronize()
        assert all(torch.equal(t, w) for t, w in zip(outputs, want))
    torch.cuda.synchronize()


@pytest.mark.parametrize("k", [512, 1440, 32])
def test_tiles(q8, k):
    import torch

    experts, n, tokens, top_k = 8, 640, 500, 2
    g = np.random.default_rng(k)
    blobs = [ref.weights_of(g, experts, n, k)[0] for _ in range(2)]
    offsets, rows = ref.groups(g, experts, tokens, top_k, "spread")
    qs, ds, _ = ref.plane_of(g, tokens, k)
    dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    dg, du, dq, dd, do, dr = dev(blobs[0]), dev(blobs[1]), dev(qs), dev(ds), dev(offsets, np.int32), dev(rows, np.int32)
    y = torch.empty(tokens * top_k, n, device="cuda")
    qo, so = q8.empty_plane(tokens * top_k, n)

    def call():
        q8.q8_0_experts_gemm(dg, experts, n, k, dq, dd, do, y, rows=dr, top_k=top_k)
        q8.q8_0_experts_gate_up(dg, du, experts, n, k, dq, dd, do, qo, so, rows=dr, top_k=top_k)

    beside_copies(call, [y, qo, so])
    q8.q8_check()


@pytest.mark.parametrize("d,top_k", [(3584, 0), (3584, 4), (7168, 1), (544, 2)])
def test_norms(q8, d, top_k):
    import torch

    rows = 700
    gen = torch.Generator("cuda").manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, b, w, h, y = r(rows, d), r(rows, d), r(d), r(rows, d), r(rows, d)
    kw = {}
    if top_k:
        kw = dict(expert_rows=r(rows * top_k, d), weights=r(rows, top_k),
                  places=torch.randperm(rows * top_k, generator=gen, device="cuda").int().view(rows, top_k))

    def call():
        q8.rmsnorm_residual_quant(x, h, b=b, w_post=w, eps_post=1e-6, w=w, eps=1e-6, y=y, **kw)

    beside_copies(call, [h, y])
    q8.q8_check()
