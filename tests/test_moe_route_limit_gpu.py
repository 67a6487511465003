"""q8_moe_route at its limit, tokens * top_k = 2^31 - 1: the last tokens' numbers plus a chunk pass 31 bits."""
import pytest

pytestmark = pytest.mark.gpu


def test_most_tokens(q8):
    import torch

    tokens, step = 2 ** 31 - 1, 1 << 28
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 46 GB: one expert's logits, ids, weights, rows and places")
    logits = torch.zeros(tokens, 1, device="cuda")
    i32 = lambda *s: torch.full(s, 99, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, weights, offsets, rows, places = i32(tokens, 1), torch.zeros(tokens, 1, device="cuda"), i32(2), i32(tokens), i32(tokens, 1)
    valid = torch.tensor([tokens - 40], dtype=torch.int32, device="cuda")
    for real, v in ((tokens, None), (tokens - 40, valid)):
        q8.q8_moe_route(logits, ids, weights, offsets, rows, places, scale=0.5, valid=v)
        q8.q8_check()
        assert offsets.tolist() == [0, real]
        for t in range(0, tokens, step):
            end = min(t + step, tokens)
            at = torch.arange(t, end, dtype=torch.int32, device="cuda")
            there = at < real
            assert torch.equal(ids[t:end, 0], torch.where(there, 0, -1).int())
            assert torch.equal(weights[t:end, 0], there * 0.5)
            at = torch.where(there, at, -1)
            assert torch.equal(rows[t:end], at) and torch.equal(places[t:end, 0], at)
    del logits, ids, weights, rows, places
    torch.cuda.empty_cache()
