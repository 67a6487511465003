"""q8_moe_route where a CTA's bit sets are as large as they get: many tokens on many experts."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def route(logits, top_k):
    """ids, weights (64 bits), offsets, rows, places of a routing without equal logits in a row, on the GPU."""
    import torch

    tokens, experts = logits.shape
    top, ids = torch.topk(logits, top_k, dim=1)
    weights = torch.softmax(top.double(), 1)
    flat = ids.reshape(-1)
    rows = torch.sort(flat, stable=True).indices
    places = torch.empty_like(rows)
    places[rows] = torch.arange(rows.numel(), device="cuda")
    counts = torch.bincount(flat, minlength=experts)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), counts.cumsum(0)])
    return ids.int(), weights, offsets.int(), rows.int(), places.view(tokens, top_k).int()


# the bits and the placing kernel's sums together: the most bits of a launch are those of 1024 experts from 38913 tokens on, of 768
# from 53505, of 512 from 82689, of 384 from 111873
@pytest.mark.parametrize("tokens,experts,top_k", [(40000, 1024, 3), (53600, 768, 1), (83001, 512, 2), (112000, 384, 2), (151000, 288, 1),
                                                  (500000, 1000, 1), (300000, 4, 4)])
def test_route(q8, tokens, experts, top_k):
    import torch

    gen = torch.Generator("cuda").manual_seed(tokens)
    # a row's logits are all different: a permutation of the experts
    logits = torch.rand(tokens, experts, generator=gen, device="cuda").argsort(1).float() / 64
    full = lambda *s: torch.full(s, 99, dtype=torch.int32, device="cuda")  # noqa: E731
    out = (full(tokens, top_k), torch.full((tokens, top_k), float("nan"), device="cuda"), full(experts + 1), full(tokens * top_k),
           full(tokens, top_k))
    q8.q8_moe_route(logits, *out)
    q8.q8_check()
    ids, weights, offsets, rows, places = route(logits, top_k)
    assert torch.equal(out[0], ids) and torch.equal(out[2], offsets)
    assert torch.equal(out[3], rows) and torch.equal(out[4], places)
    # exp to 2 steps of 2^-23, a sum of up to 16, a quotient and a product: under 2^-18
    assert torch.all((out[1] - weights).abs() <= 2.0 ** -18 * weights)
