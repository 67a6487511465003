"""The operators of a mixture-of-experts block, measured: the routing, the experts' products, the block's norms.

A block of such a layer is: the router's logits choose top_k experts a token and sort the (token, expert) pairs by expert
(route); gate and up projections of every pair on its expert's Q8_0 weights, whose SwiGLU goes out as a q8_0 plane
(gate_up); the down projection of that plane (gemm); the weighted sum of a token's experts, the norm behind the block,
its gate, the scaled residual and the norm before the next block (norm).  Every case is one such call.  The plain form
computes it with elementary torch operations; with ``own`` true the framework's entry points are called instead.  Model
widths (3584, 18944), prompts of 3325 tokens and small batches of 16 are this repository's layer stack; the numbers of
experts and their narrow widths are generic.
"""
import math

import torch

own = False

EPS = 1e-6


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token decoding: pure latency
        dict(name="route_token", op="route", tokens=1, experts=64, top_k=8, chosen=True, masked=False, padded=False),
        # a whole prompt routed at once
        dict(name="route_prompt", op="route", tokens=3325, experts=128, top_k=8, chosen=True, masked=False, padded=False),
        # one token decoding: the weights of its eight experts are read once
        dict(name="gate_up_token", op="gate_up", tokens=1, experts=64, top_k=8, k=3584, n=1280),
        # a batch of decoding sequences: nearly all experts are read, a few rows each
        dict(name="gate_up_batch", op="gate_up", tokens=61, experts=64, top_k=8, k=3584, n=1280),
        # a whole prompt: hundreds of rows an expert
        dict(name="gate_up_prompt", op="gate_up", tokens=3325, experts=64, top_k=8, k=3584, n=1280),
        # the down projection of one token's eight experts
        dict(name="down_token", op="gemm", tokens=1, experts=64, top_k=8, k=1280, n=3584, gather=False),
        # a small batch on more and wider experts; a width whose rows of blocks have no common alignment
        dict(name="down_batch", op="gemm", tokens=16, experts=128, top_k=4, k=1440, n=3584, gather=False),
        # the down projection of a whole prompt
        dict(name="down_prompt", op="gemm", tokens=3325, experts=64, top_k=8, k=1280, n=3584, gather=False),
        # few experts as wide as the dense layer, a chunk of a prompt
        dict(name="up_wide", op="gemm", tokens=509, experts=8, top_k=2, k=3584, n=18944, gather=True),
        # the end of one token's block: eight expert rows joined, both norms, the next plane
        dict(name="norm_token", op="norm", rows=1, d=3584, top_k=8, dense=False, post=True, gate="channel", plane=True),
        # the end of a dense block of a whole prompt, the next block's input in f32
        dict(name="norm_prompt", op="norm", rows=3325, d=3584, top_k=0, dense=True, post=True, gate="channel", plane=False),
        # the end of an experts' block of a whole prompt: eight rows a token and a shared expert's
        dict(name="norm_join_prompt", op="norm", rows=3325, d=3584, top_k=8, dense=True, post=True, gate="channel",
             plane=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["route", "gate_up", "gate_up", "gemm", "gemm", "norm", "norm"])
    if op == "norm":
        rows, d = log(1, 3325), 32 * log(4, 112)
        top_k = rng.choice([0, 1, 2, 4, 6, 8])
        return dict(op=op, rows=rows, d=d, top_k=top_k, dense=top_k == 0 or rng.random() < 0.4, post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "row"]), plane=rng.random() < 0.7)
    experts = rng.choice([4, 8, 16, 32, 60, 64, 128, 160])
    top_k = rng.choice([k for k in (1, 2, 4, 6, 8) if k <= experts])
    if op == "route":
        return dict(op=op, tokens=log(1, 8192), experts=experts, top_k=top_k, chosen=rng.random() < 0.6,
                    masked=rng.random() < 0.3, padded=rng.random() < 0.3)
    k = 256 * log(1, 14) if rng.random() < 0.6 else 32 * log(4, 112)
    n = 32 * log(2, 80) if op == "gate_up" else log(33, 3584)
    room = 600_000_000 // (n * k * (2 if op == "gate_up" else 1))  # weights of all experts
    experts = max(top_k, min(experts, room))
    most = 100_000_000_000 // (top_k * n * k * (2 if op == "gate_up" else 1))
    tokens = log(1, max(2, min(4096, most)))
    case = dict(op=op, tokens=tokens, experts=experts, top_k=top_k, k=k, n=n)
    return case if op == "gate_up" else dict(case, gather=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------
def encode(x):
    """f32 rows -> the q8_0 plane's codes and block scales (f32, before they are stored as f16)."""
    v = x.view(*x.shape[:-1], -1, 32)
    d = v.abs().amax(-1) / torch.full((), 127.0, dtype=x.dtype, device=x.device)
    inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
    return torch.round(v * inv[..., None]).clamp(-127, 127), d


def plane_of(x):
    """(qs int8 [rows_pad][k], ds int32 [rows_pad][k/32]: f16 scale and int16 block sum), rows padded to 128."""
    rows, k = x.shape
    pad = -(-rows // 128) * 128
    q, d = encode(x)
    qs = torch.zeros(pad, k, dtype=torch.int8, device="cuda")
    ds = torch.zeros(pad, k // 32, dtype=torch.int32, device="cuda")
    qs[:rows] = q.view(rows, k).to(torch.int8)
    bits = d.half().view(torch.int16).to(torch.int32) & 0xffff
    ds[:rows] = bits | (q.sum(-1).to(torch.int32) << 16)
    return qs, ds


def q8_weights(experts, n, k, gen):
    """uint8 [experts][n][k/32][34]: little-endian f16 scale, then 32 int8 codes."""
    shape = (experts, n, k // 32)
    codes = torch.empty(*shape, 32, dtype=torch.float16, device="cuda").normal_(generator=gen).mul_(40).clamp_(-127, 127)
    d = torch.empty(*shape, 1, device="cuda").uniform_(0.5, 1.5, generator=gen) / (40 * math.sqrt(k))
    return torch.cat([d.half().view(torch.uint8), codes.to(torch.int8).view(torch.uint8)], -1)


def logits_of(tokens, experts, gen):
    """Router logits: a token's own preferences and the experts' unequal popularity."""
    x = torch.randn(tokens, experts, generator=gen, device="cuda")
    return x + 0.4 * torch.randn(experts, generator=gen, device="cuda")


def sort_pairs(ids, experts):
    """ids [tokens][top_k] (-1: none) -> offsets [experts + 1], rows [pairs], places [tokens][top_k], as the routing defines
    them: pairs by expert, then by token; behind the last one -1."""
    flat = torch.where(ids >= 0, ids, experts).reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = (flat[:, None] == torch.arange(experts, device=flat.device)).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=flat.device), torch.cumsum(counts, 0)])
    at = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(at < offsets[-1], order, -1)
    places = torch.empty_like(order)
    places[order] = at
    places = torch.where(flat < experts, places, -1)
    return offsets.int(), rows.int(), places.view(ids.shape).int()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op == "norm":
        rows, d, top_k = case["rows"], case["d"], case["top_k"]

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        s["x"] = randn(rows, d) * 4
        s["b"] = randn(rows, d) if case["dense"] else None
        s["ye"] = s["places"] = s["weights"] = None
        if top_k:
            s["ye"] = randn(rows * top_k, d)
            s["places"] = torch.randperm(rows * top_k, generator=gen, device="cuda").int().view(rows, top_k)
            s["weights"] = torch.softmax(randn(rows, top_k), -1)
        s["w_post"] = 1 + 0.2 * randn(d) if case["post"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: 0.3 * randn(1, d), "row": lambda: 0.3 * randn(rows, d)}[case["gate"]]()
        s["w"] = 1 + 0.2 * randn(d)
        s["h"] = torch.zeros(rows, d, device="cuda")
        pad = -(-rows // 128) * 128
        if case["plane"]:
            s["qs"] = torch.zeros(pad, d, dtype=torch.int8, device="cuda")
            s["ds"] = torch.zeros(pad, d // 32, dtype=torch.int32, device="cuda")
        else:
            s["y"] = torch.zeros(rows, d, device="cuda")
        return s
    tokens, experts, top_k = case["tokens"], case["experts"], case["top_k"]
    logits = logits_of(tokens, experts, gen)
    if op == "route":
        logits = torch.round(logits * 4096) / 4096  # a router's coarse logits: equal ones occur
        if case["masked"]:  # experts that a token must not use, sometimes all but a few
            share = torch.rand(tokens, 1, generator=gen, device="cuda")
            logits[torch.rand(tokens, experts, generator=gen, device="cuda") < share] = -math.inf
        s["logits"] = logits
        real = int(tokens * 0.8) if case["padded"] else tokens
        s["valid"] = torch.tensor([real], dtype=torch.int32).cuda() if case["padded"] else None
        s["ids"] = torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros(tokens, top_k, device="cuda")
        s["offsets"] = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        s["rows"] = torch.zeros(tokens * top_k, dtype=torch.int32, device="cuda")
        s["places"] = torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda")
        return s
    ids = torch.topk(logits, top_k, dim=-1).indices
    s["offsets"], s["rows"], _ = sort_pairs(ids, experts)
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    k, n, pairs = case["k"], case["n"], tokens * top_k
    gather = op == "gate_up" or case["gather"]
    x = torch.randn(tokens if gather else pairs, k, generator=gen, device="cuda")
    x[:, ::61] *= 6.0  # outlier channels, as activations have them
    s["qs"], s["ds"] = plane_of(x)
    if op == "gate_up":
        s["w_gate"], s["w_up"] = q8_weights(experts, n, k, gen), q8_weights(experts, n, k, gen)
        s["qs_out"] = torch.zeros(-(-pairs // 128) * 128, n, dtype=torch.int8, device="cuda")
        s["ds_out"] = torch.zeros(-(-pairs // 128) * 128, n // 32, dtype=torch.int32, device="cuda")
    else:
        s["w"] = q8_weights(experts, n, k, gen)
        s["y"] = torch.zeros(pairs, n, device="cuda")
        if not gather:
            s["rows"] = None
    return s


# ----------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------------------------------------------------
def values(qs, ds, rows):
    """The numbers that a plane's first rows stand for, as f16 like the plane's scales."""
    d = ds[:rows].view(torch.float16)[:, ::2]
    return (qs[:rows].view(rows, -1, 32) * d[:, :, None]).view(rows, -1)


def run_own(s):
    import int8_quantized_projection_gb300 as q8

    case = s["case"]
    op = case["op"]
    if op == "route":
        q8.q8_moe_route(s["logits"], s["ids"], s["weights"], s["offsets"], s["rows"], s["places"],
                        mode=q8.ROUTE_CHOSEN if case["chosen"] else q8.ROUTE_ALL, valid=s["valid"])
        return {key: s[key] for key in ("ids", "weights", "offsets", "rows", "places")}
    if op == "norm":
        q8.rmsnorm_residual_quant(s["x"], s["h"], b=s["b"], expert_rows=s["ye"], places=s["places"], weights=s["weights"],
                                  w_post=s["w_post"], eps_post=EPS, gate=s["gate"], residual_scale=0.75, w=s["w"], eps=EPS,
                                  y=s.get("y"), qs=s.get("qs"), ds=s.get("ds"))
        return {"h": s["h"], "y": values(s["qs"], s["ds"], case["rows"]) if case["plane"] else s["y"]}
    if op == "gate_up":
        q8.q8_0_experts_gate_up(s["w_gate"], s["w_up"], case["experts"], case["n"], case["k"], s["qs"], s["ds"],
                                s["offsets"], s["qs_out"], s["ds_out"], rows=s["rows"], top_k=case["top_k"])
        return values(s["qs_out"], s["ds_out"], case["tokens"] * case["top_k"])
    q8.q8_0_experts_gemm(s["w"], case["experts"], case["n"], case["k"], s["qs"], s["ds"], s["offsets"], s["y"],
                         rows=s["rows"], top_k=case["top_k"])
    return s["y"]


# ----------------------------------------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------------------------------------
def route_plain(s):
    case, logits = s["case"], s["logits"]
    tokens, experts = logits.shape
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)  # equal logits: the lower expert first
    top, ids = best[:, :case["top_k"]], ids[:, :case["top_k"]]
    fine = top > -math.inf
    if s["valid"] is not None:
        fine = fine & (torch.arange(tokens, device="cuda") < s["valid"])[:, None]
    first = torch.where(top[:, :1] > -math.inf, top[:, :1], 0.0)
    e = torch.where(fine, torch.exp(top - first), 0.0)
    total = e.sum(-1, keepdim=True) if case["chosen"] else torch.exp(logits - first).sum(-1, keepdim=True)
    s["weights"].copy_(torch.where(fine, e / total, 0.0))
    ids = torch.where(fine, ids, -1)
    s["ids"].copy_(ids)
    offsets, rows, places = sort_pairs(ids, experts)
    s["offsets"].copy_(offsets), s["rows"].copy_(rows), s["places"].copy_(places)
    return {key: s[key] for key in ("ids", "weights", "offsets", "rows", "places")}


def norm_plain(s):
    case, x = s["case"], s["x"]
    b = s["b"]
    if s["ye"] is not None:
        join = (s["ye"][s["places"].long()] * s["weights"][:, :, None]).sum(1)
        b = join if b is None else b + join
    if s["w_post"] is not None:
        b = b * torch.rsqrt((b * b).mean(-1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        b = b * s["gate"]
    h = 0.75 * x + b
    s["h"].copy_(h)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    if not case["plane"]:
        s["y"].copy_(y)
        return {"h": s["h"], "y": s["y"]}
    q, d = encode(y)
    return {"h": s["h"], "y": (q.half() * d.half()[..., None]).view(y.shape)}


def widen(blocks):
    """Q8_0 blocks [...][n][k/32][34] -> f32 [...][n][k]."""
    d = blocks[..., :2].contiguous().view(torch.float16).float()
    return (blocks[..., 2:].view(torch.int8).float() * d).flatten(-2)


def activations(s):
    """The plane's values in the order of the sorted pairs, and each pair's expert."""
    case = s["case"]
    pairs = case["tokens"] * case["top_k"]
    at = torch.arange(pairs, device="cuda")
    rows = at if s["rows"] is None else s["rows"].long() // case["top_k"]
    d = s["ds"].view(torch.float16)[:, ::2].float()
    x = (s["qs"].view(s["qs"].shape[0], -1, 32).float() * d[:, :, None]).flatten(1)[rows]
    return x, torch.searchsorted(s["offsets"][1:].long().contiguous(), at, right=True)


def product_plain(s, x, expert, blocks):
    experts = s["case"]["experts"]
    if x.shape[0] <= experts:  # few pairs: the weights of their experts alone
        return torch.bmm(widen(blocks[expert]), x[:, :, None])[:, :, 0]
    # else every expert's rows padded to the longest
    node = torch.arange(x.shape[0], device="cuda") - s["offsets"].long()[expert]
    padded = torch.zeros(experts, s["most"], x.shape[1], device="cuda")
    padded[expert, node] = x
    return torch.bmm(padded, widen(blocks).transpose(1, 2))[expert, node]


def gate_up_plain(s):
    x, expert = activations(s)
    g, u = product_plain(s, x, expert, s["w_gate"]), product_plain(s, x, expert, s["w_up"])
    q, d = encode(g / (1 + torch.exp(-g)) * u)
    return (q.half() * d.half()[..., None]).flatten(1)


def gemm_plain(s):
    x, expert = activations(s)
    s["y"].copy_(product_plain(s, x, expert, s["w"]))
    return s["y"]


def run(state):
    if own:
        return run_own(state)
    return {"route": route_plain, "gate_up": gate_up_plain, "gemm": gemm_plain, "norm": norm_plain}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "norm":
        size = case["rows"] * case["d"]
        reads = 1 + case["top_k"] + case["dense"] + (case["gate"] == "row")
        out = 4 + (1.125 if case["plane"] else 4)
        return {"bytes": size * (4 * reads + out), "flops": size * (2 * case["top_k"] + 10)}
    tokens, experts, top_k = case["tokens"], case["experts"], case["top_k"]
    pairs = tokens * top_k
    if op == "route":
        return {"bytes": 4 * (tokens * experts + 4 * pairs + experts), "flops": tokens * experts * 2}
    k, n = case["k"], case["n"] * (2 if op == "gate_up" else 1)
    used = experts * (1 - (1 - top_k / experts) ** tokens)  # experts that some token chose
    rows_in = tokens if op == "gate_up" or case["gather"] else pairs
    out = pairs * case["n"] * (1.125 if op == "gate_up" else 4)
    return {"bytes": used * n * k * 34 / 32 + rows_in * k * 1.125 + out + 4 * pairs, "flops": 2 * pairs * n * k}


# ----------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------------------
def coded(y):
    """What the q8_0 encoding of y [rows][k] stands for, in 64 bits but for the scale, which is stored as f16."""
    v = y.reshape(y.shape[0], -1, 32)
    d = v.abs().max(-1, keepdim=True).values / 127
    code = torch.where(d > 0, torch.round(v / d), torch.zeros_like(v))
    return (code * d.half().double()).reshape(y.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        logits = s["logits"].double()
        real = logits.shape[0] if s["valid"] is None else int(s["valid"])
        p = torch.softmax(logits, -1).nan_to_num(0.0)  # a token whose logits are all -inf has no expert
        top = torch.sort(p, -1, descending=True).values[:, :case["top_k"]]
        if case["chosen"]:
            top = (top / top.sum(-1, keepdim=True)).nan_to_num(0.0)
        top[real:] = 0
        return {"ids": None, "weights": top, "offsets": None, "rows": None, "places": None}
    if op == "norm":
        b = torch.zeros_like(s["x"], dtype=torch.float64)
        if s["b"] is not None:
            b += s["b"]
        for j in range(case["top_k"]):
            b += s["weights"][:, j:j + 1].double() * s["ye"].double().index_select(0, s["places"][:, j].long())
        if s["w_post"] is not None:
            b = b / torch.sqrt(b.square().mean(1, keepdim=True) + EPS) * s["w_post"].double()
        if s["gate"] is not None:
            b = b * s["gate"].double()
        h = s["x"].double() * 0.75 + b
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].double()
        return {"h": h, "y": coded(y) if case["plane"] else y}
    tokens, top_k, n, k = case["tokens"], case["top_k"], case["n"], case["k"]
    pairs = tokens * top_k
    if pairs * n * k * (2 if op == "gate_up" else 1) > 2.6e11:
        return None
    scale = (s["ds"] & 0xffff).to(torch.int16).view(torch.float16).double()
    x = s["qs"].double() * scale.repeat_interleave(32, 1)
    source = torch.arange(pairs, device="cuda") if s["rows"] is None else torch.div(s["rows"].long(), top_k, rounding_mode="floor")

    def product(w):
        out = torch.zeros(pairs, n, dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(case["experts"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                code = w[e, :, :, 2:].contiguous().view(torch.int8).double()
                d = w[e, :, :, 0].int() | (w[e, :, :, 1].int() << 8)
                full = code * d.to(torch.int16).view(torch.float16).double()[..., None]
                out[lo:hi] = x[source[lo:hi]] @ full.reshape(n, k).T
        return out

    if op == "gemm":
        return product(s["w"])
    g, u = product(s["w_gate"]), product(s["w_up"])
    return coded(g * torch.sigmoid(g) * u)
