"""q8_kv_plan and q8_kv_accept refuse an output in an input's place: other CTAs still read what the first ones would
overwrite.  Addresses are never dereferenced: every call is refused, or finds no GPU."""
import ctypes

import pytest
import torch

import int8_quantized_projection_gb300 as q8p
from int8_quantized_projection_gb300 import build

from .test_kv_abi_host import desc, ref

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses reach no GPU")

P = ctypes.c_void_p
ERR_ARG, ERR_DEVICE = 1, 3
BATCH, PAGES, TOKENS, WIDTH = 2, 4, 6, 8
STEP = 0x1000  # between the arrays


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q8p.lib()


# name -> bytes
PLAN = dict(cached=BATCH * 4, fresh=BATCH * 4, held=BATCH * 4, free=4 * 4, table=BATCH * PAGES * 4, parents=TOKENS * 4,
            starts=(BATCH + 1) * 4, slots=TOKENS * 4, positions=TOKENS * 4, masks=TOKENS * 8, needed=4, held_out=BATCH * 4)
PLAN_OUT = ("table", "starts", "slots", "positions", "masks", "needed", "held_out")
ACCEPT = dict(table=BATCH * PAGES * 4, cached=BATCH * 4, fresh=BATCH * 4, paths=BATCH * WIDTH * 4, counts=BATCH * 4,
              lens=BATCH * 4)


def apart(sizes):
    return {n: 0x10000 + STEP * i for i, n in enumerate(sizes)}


def plan(lib, p):
    return lib.q8_kv_plan(P(p["cached"]), P(p["fresh"]), BATCH, P(p["held"]), P(p["free"]), 4, P(p["table"]), PAGES, 16, 8,
                          P(p["parents"]), TOKENS, P(p["starts"]), P(p["slots"]), P(p["positions"]), P(p["masks"]),
                          P(p["needed"]), P(p["held_out"]), P(0))


def accept(lib, p):
    return lib.q8_kv_accept(ref(desc()), P(p["table"]), PAGES, P(p["cached"]), P(p["fresh"]), BATCH, P(p["paths"]),
                            P(p["counts"]), WIDTH, P(p["lens"]), P(0))


@pytest.mark.parametrize("out,other", [(a, b) for a in PLAN_OUT for b in PLAN if a != b])
def test_plan(lib, out, other):
    p = apart(PLAN)
    p[out] = p[other]
    assert plan(lib, p) == ERR_ARG
    p[out] = p[other] + (PLAN[other] - 4 & ~15)  # the last bytes only
    assert plan(lib, p) == ERR_ARG
    p[out] = p[other] + (PLAN[other] + 15 & ~15)  # right behind
    assert plan(lib, p) == ERR_DEVICE


@pytest.mark.parametrize("other", [n for n in ACCEPT if n != "lens"])
def test_accept(lib, other):
    p = apart(ACCEPT)
    p["lens"] = p[other]
    assert accept(lib, p) == ERR_ARG
    p["lens"] = p[other] + (ACCEPT[other] - 4 & ~15)
    assert accept(lib, p) == ERR_ARG
    p["lens"] = p[other] + (ACCEPT[other] + 15 & ~15)
    assert accept(lib, p) == ERR_DEVICE


def test_missing_arrays_overlap_nothing(lib):
    p = apart(PLAN)
    for n in ("held", "parents", "masks", "held_out"):
        p[n] = 0
    assert plan(lib, p) == ERR_DEVICE
