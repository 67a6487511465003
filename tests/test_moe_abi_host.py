"""Host-side checks of the mixture-of-experts entry points: bad arguments are refused before any device work."""
import ctypes

import pytest

import int8_quantized_projection_gb300 as q8p
from int8_quantized_projection_gb300 import build

P = ctypes.c_void_p
ERR_ARG, ERR_ALIGN = 1, 2
AT = {name: (i + 1) << 40 for i, name in enumerate(
    ("logits", "valid", "ids", "weights", "offsets", "rows", "places", "ws", "w", "w2", "qs", "ds", "y", "qo", "do", "x", "b", "ye",
     "post", "gate", "h"))}  # far apart, never dereferenced: every call below fails validation first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q8p.lib()


def route(lib, tokens=500, experts=64, top_k=8, mode=1, scale=1.0, nbytes=1 << 30, **kw):
    a = {**AT, "valid": 0, **kw}
    return lib.q8_moe_route(P(a["logits"]), tokens, experts, top_k, mode, scale, P(a["valid"]), P(a["ids"]), P(a["weights"]),
                            P(a["offsets"]), P(a["rows"]), P(a["places"]), P(a["ws"]), nbytes, P(0))


def gemm(lib, experts=8, n=64, k=256, plane_rows=10, top_k=2, pairs=20, nbytes=1 << 40, **kw):
    a = {**AT, **kw}
    return lib.q8_0_experts_gemm(P(a["w"]), experts, n, k, P(a["qs"]), P(a["ds"]), plane_rows, P(a["offsets"]), P(a["rows"]),
                                 top_k, pairs, P(a["y"]), P(a["ws"]), nbytes, P(0))


def gate_up(lib, experts=8, n=64, k=256, plane_rows=10, top_k=2, pairs=20, nbytes=1 << 40, **kw):
    a = {**AT, **kw}
    return lib.q8_0_experts_gate_up(P(a["w"]), P(a["w2"]), experts, n, k, P(a["qs"]), P(a["ds"]), plane_rows, P(a["offsets"]),
                                    P(a["rows"]), top_k, pairs, P(a["qo"]), P(a["do"]), P(a["ws"]), nbytes, P(0))


def norm(lib, alpha=1.0, count=20, top_k=2, eps_post=1e-6, gate_rows=1, eps=1e-6, rows=10, d=256, rows_pad=128, **kw):
    a = {**AT, **kw}
    return lib.rmsnorm_residual_quant(P(a["x"]), alpha, P(a["b"]), P(a["ye"]), count, P(a["places"]), P(a["weights"]), top_k,
                                      P(a["post"]), eps_post, P(a["gate"]), gate_rows, P(a["w"]), eps, P(a["h"]), P(a["y"]), rows,
                                      d, P(a["qs"]), P(a["ds"]), rows_pad, P(0))


def misaligned(lib, call, names):
    for name in names:
        assert call(lib, **{name: AT[name] + 4}) == ERR_ALIGN, name


def overlapping(lib, call, pairs):
    for out, other in pairs:
        assert call(lib, **{out: AT[other]}) == ERR_ARG, (out, other)


def test_route_arguments(lib):
    for name in ("logits", "ids", "weights", "offsets", "rows", "places"):
        assert route(lib, **{name: 0}) == ERR_ARG, name
    for kw in (dict(tokens=0), dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=17),
               dict(top_k=8, experts=7), dict(mode=0), dict(mode=3), dict(scale=NAN), dict(scale=INF), dict(tokens=1 << 28),
               dict(ws=0), dict(nbytes=15)):
        assert route(lib, **kw) == ERR_ARG, kw
    misaligned(lib, route, ("logits", "valid", "ids", "weights", "offsets", "rows", "places", "ws"))
    overlapping(lib, route, [("ids", "logits"), ("ids", "rows"), ("weights", "places"), ("ws", "logits"), ("offsets", "ws")])


def test_route_workspace(lib):
    size = lib.q8_moe_route_workspace_bytes
    assert size(1, 64, 8) == 0 and size(64, 64, 8) == 0 and size(65, 64, 8) > 0
    assert size(0, 64, 8) == 0 and size(500, 64, 65) == 0 and size(500, 2000, 8) == 0
    assert size(3325, 128, 8) == 104 * 128 * 4  # chunks of 32 tokens


@pytest.mark.parametrize("call", [gemm, gate_up])
def test_product_arguments(lib, call):
    names = ["w", "qs", "ds", "offsets"] + (["y"] if call is gemm else ["w2", "qo", "do"])
    for name in names:
        assert call(lib, **{name: 0}) == ERR_ARG, name
    for kw in (dict(experts=0), dict(experts=1025), dict(n=0), dict(n=(1 << 22) + 32), dict(k=0), dict(k=16), dict(k=272),
               dict(k=(1 << 20) + 32), dict(experts=1024, n=1 << 21), dict(plane_rows=0), dict(plane_rows=1 << 31), dict(top_k=0),
               dict(top_k=17), dict(pairs=0), dict(pairs=1 << 31)):
        assert call(lib, **kw) == ERR_ARG, kw
    misaligned(lib, call, names + ["rows"])
    out = "y" if call is gemm else "qo"
    overlapping(lib, call, [(out, name) for name in ("w", "qs", "ds", "offsets", "rows")])


def test_gate_up_width(lib):
    assert gate_up(lib, n=48) == ERR_ARG
    assert lib.q8_0_experts_gate_up_workspace_bytes(8, 48, 256, 10, 2, 20) == 0


def test_workspaces_too_short(lib):
    sizes = (8, 64, 256, 10, 2, 20)
    need = lib.q8_0_experts_gate_up_workspace_bytes(*sizes)
    assert need == 0 or gate_up(lib, nbytes=need - 1) == ERR_ARG and gate_up(lib, ws=0) == ERR_ARG
    many = dict(experts=2, n=512, k=512, plane_rows=4096, top_k=1, pairs=4096)
    for call, name in ((gemm, "gemm"), (gate_up, "gate_up")):
        need = getattr(lib, f"q8_0_experts_{name}_workspace_bytes")(*many.values())
        assert need == 0 or call(lib, nbytes=need - 1, **many) == ERR_ARG and call(lib, ws=0, **many) == ERR_ARG


def test_norm_arguments(lib):
    plane = dict(qs=AT["qs"], ds=AT["ds"])
    for kw in (dict(x=0), dict(b=0, ye=0, places=0, weights=0, top_k=0), dict(d=0), dict(d=48), dict(d=32800), dict(rows=-1),
               dict(rows_pad=9), dict(qs=0), dict(ds=0), dict(w=0), dict(h=0, y=0, qs=0, ds=0, w=0), dict(h=0, y=0, qs=0, ds=0),
               dict(y=0, qs=0, ds=0), dict(ye=0), dict(places=0), dict(weights=0), dict(top_k=0), dict(top_k=17), dict(top_k=-1),
               dict(count=0), dict(count=1 << 31), dict(gate_rows=2), dict(gate_rows=0), dict(alpha=NAN), dict(alpha=INF),
               dict(eps=-1.0), dict(eps=NAN), dict(eps_post=-1.0), dict(eps_post=NAN), dict(rows=0, rows_pad=0)):
        assert norm(lib, **{**plane, **kw}) == ERR_ARG, kw
    misaligned(lib, norm, ("x", "b", "ye", "places", "weights", "post", "gate", "w", "h", "y", "qs", "ds"))
    overlapping(lib, norm, [("h", "b"), ("h", "ye"), ("y", "x"), ("y", "h"), ("qs", "x"), ("ds", "qs"), ("h", "gate"), ("y", "w")])
    assert norm(lib, h=AT["x"] + 1024) == ERR_ARG  # x itself, or apart from it


@pytest.mark.parametrize("name", ["q8_moe_route", "q8_0_experts_gemm", "q8_0_experts_gate_up", "rmsnorm_residual_quant"])
def test_python_names(name):
    assert callable(getattr(q8p, name))
