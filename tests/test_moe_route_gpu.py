"""q8_moe_route against its definition: ties, masked logits, padded batches, one launch and two."""
import numpy as np
import pytest

from tests import _moe_ref as ref

pytestmark = pytest.mark.gpu


def outputs(tokens, experts, top_k):
    import torch

    full = lambda *s: torch.full(s, 99, dtype=torch.int32, device="cuda")  # noqa: E731
    return (full(tokens, top_k), torch.full((tokens, top_k), float("nan"), device="cuda"), full(experts + 1),
            full(tokens * top_k), full(tokens, top_k))


def check(got, want):
    ids, weights, offsets, rows, places = (t.cpu().numpy() for t in got)
    assert np.array_equal(ids, want[0]) and np.array_equal(offsets, want[2])
    assert np.array_equal(rows, want[3]) and np.array_equal(places, want[4])
    # exp to 2 steps of 2^-23, a sum of up to 1024 in chains of at most 32 + 5, a quotient and a product
    assert np.all(np.abs(weights - want[1]) <= 2.0 ** -18 * np.abs(want[1]) + 1e-37)


def logits_of(g, tokens, experts, kind):
    x = g.standard_normal((tokens, experts)).astype(np.float32) * 2
    if kind == "ties":
        x = np.round(x)  # a handful of values, -0 and +0 among them
        x[g.random(x.shape) < 0.2] = -0.0
    elif kind == "masked":
        x[g.random(x.shape) < np.linspace(0, 1, tokens)[:, None]] = -np.inf
        x[g.random(x.shape) < 0.05] = np.nan
        if tokens > 2:
            x[tokens // 2] = -np.inf  # a token without any expert
            x[0, ::2] = np.inf
    return x


@pytest.mark.parametrize("kind", ["plain", "ties", "masked"])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 64, 8), (2, 3, 3), (33, 60, 4), (128, 128, 8), (129, 16, 2),
                                                  (500, 257, 16), (1000, 1024, 6), (4999, 40, 1)])
@pytest.mark.parametrize("mode", [1, 2])
def test_route(q8, tokens, experts, top_k, mode, kind):
    import torch

    g = np.random.default_rng([tokens, experts, top_k, mode])
    x = logits_of(g, tokens, experts, kind)
    out = outputs(tokens, experts, top_k)
    q8.q8_moe_route(torch.from_numpy(x).cuda(), *out, mode=mode, scale=1.5)
    q8.q8_check()
    check(out, ref.route(x, top_k, mode, 1.5))


@pytest.mark.parametrize("tokens", [7, 300])
def test_padded_batch(q8, tokens):
    import torch

    g = np.random.default_rng(5)
    x = logits_of(g, tokens, 32, "plain")
    x[-1] = np.nan  # what padding may hold
    for valid, real in ((0, 0), (1, 1), (tokens - 2, tokens - 2), (tokens, tokens)):
        out = outputs(tokens, 32, 4)
        q8.q8_moe_route(torch.from_numpy(x).cuda(), *out, valid=torch.tensor([valid], dtype=torch.int32, device="cuda"))
        q8.q8_check()
        check(out, ref.route(x, 4, 1, valid=real))
    for valid, real in ((-3, 0), (tokens + 1, tokens)):
        out = outputs(tokens, 32, 4)
        q8.q8_moe_route(torch.from_numpy(x).cuda(), *out, valid=torch.tensor([valid], dtype=torch.int32, device="cuda"))
        with pytest.raises(q8.Q8Error, match="DATA"):
            q8.q8_check()
        check(out, ref.route(x, 4, 1, valid=real))


def test_far_apart_logits(q8):
    import torch

    x = np.array([[3e38, -3e38, 1e-45, 0.0, -1e-45, 88.0], [-200.0, -100.0, -104.0, -3e38, -190.0, -100.0]], np.float32)
    out = outputs(2, 6, 5)
    q8.q8_moe_route(torch.from_numpy(x).cuda(), *out, mode=2)
    q8.q8_check()
    check(out, ref.route(x, 5, 2))


def test_refusals(q8):
    import torch

    x = torch.zeros(4, 8, device="cuda")
    out = outputs(4, 8, 2)
    for i, bad in ((0, out[0][:, :1].contiguous()), (1, out[1].double()), (2, out[2][:8]), (3, out[3][:7]), (4, out[4].long())):
        with pytest.raises(ValueError):
            q8.q8_moe_route(x, *out[:i], bad, *out[i + 1:])
    with pytest.raises(ValueError):
        q8.q8_moe_route(x.t(), *outputs(8, 4, 2))
    with pytest.raises(q8.Q8Error, match="ARG"):
        q8.q8_moe_route(x, *out, mode=7)
    with pytest.raises(q8.Q8Error, match="ARG"):
        q8.q8_moe_route(x, out[0], out[1], out[2], out[0].view(-1), out[4])
