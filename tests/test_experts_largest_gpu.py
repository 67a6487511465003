"""The experts' products at the largest numbers of experts, columns and rows that a call takes."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu


def check(q8, experts, n, k, tokens, top_k, gate_up=True):
    import torch

    g = np.random.default_rng([experts, n, k, tokens])
    (bg, wg), (bu, wu) = (ref.weights_of(g, experts, n, k) for _ in range(2))
    offsets, rows = ref.groups(g, experts, tokens, top_k, "skew" if experts > 1 else "spread")
    qs, ds, x = ref.plane_of(g, tokens, k)
    dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    dg, du, dq, dd, do, dr = dev(bg), dev(bu), dev(qs), dev(ds), dev(offsets, np.int32), dev(rows, np.int32)
    pairs = tokens * top_k
    y = torch.full((pairs, n), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(dg, experts, n, k, dq, dd, do, y, rows=dr, top_k=top_k)
    gt, gl = ref.product(wg, x, offsets, rows // top_k)
    assert np.all(np.abs(y.cpu().numpy() - gt) <= gl)
    if gate_up:
        qo, so = q8.empty_plane(pairs, n)
        q8.q8_0_experts_gate_up(dg, du, experts, n, k, dq, dd, do, qo, so, rows=dr, top_k=top_k)
        ref.check_plane(qo.cpu().numpy(), so.cpu().numpy(), *ref.swiglu(gt, gl, *ref.product(wu, x, offsets, rows // top_k)))
    q8.q8_check()


@pytest.mark.parametrize("k", [256, 96])
@pytest.mark.parametrize("tokens,top_k", [(3, 2), (300, 16), (1000, 16), (1700, 16)])
def test_1024_experts(q8, tokens, top_k, k):
    """A few rows on some of them, eight and sixteen rows a segment, tiles; most pairs on few experts."""
    check(q8, 1024, 32, k, tokens, top_k)


LONGEST = pytest.mark.parametrize("k", [1 << 20, (1 << 20) - 32])
FEW = pytest.mark.parametrize("experts,tokens", [(2, 3), (1, 12), (1, 40)])


@FEW
@LONGEST
def test_longest_rows(q8, experts, tokens, k):
    """The gemm alone: of 32768 blocks of any sign the limit, 32776 * 2^-24 of the sum of magnitudes, is as large as the sums."""
    check(q8, experts, 32, k, tokens, 1, gate_up=False)


@FEW
@LONGEST
def test_longest_rows_exactly(q8, experts, tokens, k):
    """Codes up to 3 and scales that are powers of two: every partial sum is an integer up to 2^20 * 9 < 2^24 times a power of two,
    so f32 has it exactly in any order, and the plane is swiglu_quant's of the exact products."""
    import torch

    n = 64
    g = np.random.default_rng([experts, tokens, k])
    scale = lambda e: np.float16(2.0 ** e).view(np.uint16)  # noqa: E731
    codes = [g.integers(-3, 4, (experts, n, k)).astype(np.int8) for _ in range(2)]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    blobs = []
    for c in codes:
        b = np.empty((experts * n, k // 32, 34), np.uint8)
        b[..., :2] = np.frombuffer(scale(-6).tobytes(), np.uint8)
        b[..., 2:] = c.reshape(experts * n, k // 32, 32).view(np.uint8)
        blobs.append(dev(b.reshape(-1)))
    q = g.integers(-3, 4, (tokens, k)).astype(np.int8)
    dq, dd = dev(q), torch.full((tokens, k // 32), int(scale(-8)), dtype=torch.int32, device="cuda")
    offsets = np.linspace(0, tokens, experts + 1).astype(np.int32)
    do = dev(offsets)
    y = [torch.full((tokens, n), float("nan"), device="cuda") for _ in range(2)]
    for w, o in zip(blobs, y):
        q8.q8_0_experts_gemm(w, experts, n, k, dq, dd, do, o)
    plane, want = q8.empty_plane(tokens, n), q8.empty_plane(tokens, n)
    q8.q8_0_experts_gate_up(*blobs, experts, n, k, dq, dd, do, *plane)
    for c, o in zip(codes, y):
        for e in range(experts):
            rows = slice(offsets[e], offsets[e + 1])
            exact = q[rows].astype(np.float64) @ c[e].T.astype(np.float64) * 2.0 ** -14
            assert np.array_equal(o[rows].cpu().numpy(), exact)
    q8.swiglu_quant(*y, None, *want)
    q8.q8_check()
    assert torch.equal(plane[0], want[0]) and torch.equal(plane[1], want[1])


@pytest.mark.parametrize("tokens", [3, 30])
def test_most_rows_of_a_matrix(q8, tokens):
    """n = 2^22: an expert's outputs against 64 bits on the GPU."""
    import torch

    n, k = 1 << 22, 32
    gen = torch.Generator("cuda").manual_seed(tokens)
    codes = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    d = torch.rand(n, 1, generator=gen, device="cuda").half()
    w = torch.cat([d.view(torch.uint8).view(n, 2), codes.view(torch.uint8)], 1).contiguous()
    qs = torch.randint(-127, 128, (tokens, k), generator=gen, device="cuda", dtype=torch.int8)
    da = torch.rand(tokens, 1, generator=gen, device="cuda").half()
    ds = da.view(torch.int16).int() & 0xffff
    offsets = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    y = torch.full((tokens, n), float("nan"), device="cuda")
    q8.q8_0_experts_gemm(w.view(-1), 1, n, k, qs, ds, offsets, y)
    qo, so = q8.empty_plane(tokens, n)
    q8.q8_0_experts_gate_up(w.view(-1), w.view(-1), 1, n, k, qs, ds, offsets, qo, so)
    q8.q8_check()
    full = codes.double() * d.double()
    for t in range(tokens):
        want = full @ (qs[t].double() * da[t].double())
        assert torch.all((y[t] - want).abs() <= 2.0 ** -22 * want.abs())  # one product of two exact factors
    qw, sw = q8.empty_plane(tokens, n)
    q8.swiglu_quant(y, y, None, qw, sw)
    assert torch.equal(qo, qw) and torch.equal(so, sw)
