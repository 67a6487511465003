"""q8_check: every error word is read and cleared, from any stream and from several threads, without a copy for each."""
import statistics
import threading
import time

import numpy as np
import pytest

from . import _kv_ref as ref

pytestmark = pytest.mark.gpu


def bad_append(q8):
    import torch

    cache = q8.empty_kv_cache(1, 2, 1, 16, 64)
    x = torch.randn(1, 64, device="cuda")
    q8.q8_kv_append(cache, 0, x, x, torch.tensor([32], dtype=torch.int32, device="cuda"))


def bad_attention(q8, heads):
    c = ref.Case(140, [20, 5], [1, 1], heads, 1, 64, 16, False)
    c.cached[1] = -5
    c.run()


CALLS = [bad_append, lambda q8: bad_attention(q8, 4), lambda q8: bad_attention(q8, 40)]  # a word of its own each


def status(q8, stream=None):
    try:
        q8.q8_check(stream)
    except q8.Q8Error as e:
        return e.status
    return 0


@pytest.mark.parametrize("words", [[0], [1], [2], [0, 1], [2, 1, 0]])
@pytest.mark.parametrize("other", [False, True])
def test_each_word_is_reported_once(q8, words, other):
    import torch

    stream = torch.cuda.Stream() if other else None
    for w in words:
        CALLS[w](q8)
    torch.cuda.synchronize()
    assert [status(q8, stream) for _ in range(3)] == [8, 0, 0]
    assert status(q8) == 0


def test_checks_from_several_threads(q8):
    """Each error is told to one of them, and none fails."""
    import torch

    rounds, got = 20, []
    streams = [torch.cuda.Stream() for _ in range(6)]
    start = threading.Barrier(len(streams) + 1, timeout=60)

    def worker(s):
        for _ in range(rounds):
            start.wait()
            got.append(status(q8, s))
            start.wait()

    threads = [threading.Thread(target=worker, args=(s,)) for s in streams]
    for t in threads:
        t.start()
    for _ in range(rounds):
        bad_append(q8)
        torch.cuda.synchronize()
        start.wait()
        start.wait()
    for t in threads:
        t.join()
    assert sorted(got) == [0] * (rounds * (len(streams) - 1)) + [8] * rounds
    assert status(q8) == 0


def test_a_check_costs_few_round_trips(q8):
    """Timed beside a four-byte read of PyTorch's, which is one copy and one wait."""
    import torch

    x = torch.zeros(1, dtype=torch.int32, device="cuda")

    def median(f):
        took = []
        for _ in range(200):
            t = time.perf_counter()
            f()
            took.append(time.perf_counter() - t)
        return statistics.median(took[20:])

    torch.cuda.synchronize()
    assert np.median([median(q8.q8_check) / median(x.item) for _ in range(3)]) < 4.0
