"""The paged key/value cache's operators, measured: the step plan, the append, the attention of drafted tokens, the accept.

Every case is one call on what a serving loop has in hand at that moment.  The plain form computes it with elementary
torch operations; with ``own`` true the framework's entry points are called instead.  Head layouts are those of this
repository's layer stack (28 query heads and 4 key/value heads of 128, 28 layers, prompts of 3325 tokens, small
batches of 16) and generic ones.
"""
import math
import random

import torch

own = False

NODES = 64  # most drafted tokens a sequence has in a tree (one mask word)


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one sequence decoding its next token: pure latency
        dict(name="plan_one", op="plan", batch=1, cached=1000, fresh=1, page=16, tree=False),
        # a full server verifying draft trees of up to 64 nodes
        dict(name="plan_trees", op="plan", batch=509, cached=9000, fresh=64, page=64, tree=True),
        # the k and v rows of a single token
        dict(name="append_token_f16", op="append", tokens=1, kv_heads=4, dim=128, page=16, kind="f16"),
        # the k and v rows of a whole prompt, kept as int8
        dict(name="append_prompt_int8", op="append", tokens=3325, kv_heads=4, dim=128, page=64, kind="int8"),
        # single-token decode of one sequence
        dict(name="decode_one_f16", op="attention", batch=1, cached=4097, fresh=1, heads=28, kv_heads=4, dim=128, page=16,
             kind="f16", tree=False),
        # single-token decode of a batch of ragged lengths, int8 cache
        dict(name="decode_batch_int8", op="attention", batch=61, cached=8191, fresh=1, heads=28, kv_heads=4, dim=128,
             page=64, kind="int8", tree=False),
        # single-token decode over one very long context
        dict(name="decode_long_f16", op="attention", batch=1, cached=262139, fresh=1, heads=28, kv_heads=4, dim=128,
             page=128, kind="f16", tree=False),
        # trees of up to 16 drafted tokens verified over ragged contexts
        dict(name="tree16_f16", op="attention", batch=8, cached=16001, fresh=16, heads=28, kv_heads=4, dim=128, page=32,
             kind="f16", tree=True),
        # trees of up to 64 drafted tokens over an int8 cache
        dict(name="tree64_int8", op="attention", batch=4, cached=30011, fresh=64, heads=28, kv_heads=4, dim=128, page=64,
             kind="int8", tree=True),
        # a whole prompt attending to itself
        dict(name="prompt_f16", op="attention", batch=1, cached=0, fresh=3325, heads=28, kv_heads=4, dim=128, page=64,
             kind="f16", tree=False),
        # one sequence's accepted path moved to the front, every layer
        dict(name="accept_one_f16", op="accept", batch=1, cached=1000, fresh=16, layers=28, kv_heads=4, dim=128, page=16,
             kind="f16"),
        # a batch's accepted paths
        dict(name="accept_batch_int8", op="accept", batch=128, cached=300, fresh=32, layers=28, kv_heads=4, dim=128,
             page=64, kind="int8"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["plan", "append", "attention", "attention", "attention", "accept"])
    page, kind = rng.choice([16, 32, 48, 64, 128]), rng.choice(["f16", "int8"])
    heads, kv_heads = rng.choice([(28, 4), (32, 8), (16, 16), (12, 1), (8, 2), (40, 8)])
    dim = rng.choice([64, 128, 128])
    if op == "plan":
        tree = rng.random() < 0.5
        return dict(op=op, batch=log(1, 509), cached=log(1, 9000), fresh=log(1, NODES), page=page, tree=tree)
    if op == "append":
        return dict(op=op, tokens=log(1, 3325), kv_heads=kv_heads, dim=dim, page=page, kind=kind)
    if op == "accept":
        return dict(op=op, batch=log(1, 128), cached=log(1, 300), fresh=log(2, 32), layers=rng.randint(1, 28),
                    kv_heads=min(kv_heads, 4), dim=dim, page=page, kind=kind)
    form = rng.choice(["decode", "decode", "tree", "tree", "chunk"])
    if form == "chunk":  # a chunk of a prompt behind earlier chunks
        fresh = log(65, 2048)
        return dict(op=op, batch=1, cached=log(1, 2048), fresh=fresh, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    kind=kind, tree=False)
    batch = log(1, 61)
    rows = 1 if form == "decode" else log(2, NODES)
    room = 500_000 if form == "decode" else 2_000_000 // max(16, rows)  # keys of the whole batch
    cached = log(1, max(2, min(262139, room * 4 // (batch * kv_heads))))
    return dict(op=op, batch=batch, cached=cached, fresh=rows, heads=heads, kv_heads=kv_heads, dim=dim, page=page, kind=kind,
                tree=form == "tree")


# ----------------------------------------------------------------------------------------------------------------------
# lengths: ragged over the batch, the same multiset for every seed (the longest is the case's own figure)
# ----------------------------------------------------------------------------------------------------------------------
def lengths(case, seed=None):
    batch, cached, fresh = case["batch"], case["cached"], case["fresh"]
    r = random.Random(f"{batch} {cached} {fresh}")
    pairs = [(cached, fresh)]
    for _ in range(batch - 1):
        pairs.append((int(cached * r.random() ** 0.7), r.randint(0, fresh) if r.random() < 0.5 else fresh))
    if case["op"] == "accept" or (case["op"] == "attention" and fresh == 1):
        pairs = [(c, max(f, 1)) for c, f in pairs]
    if seed is not None:
        random.Random(seed).shuffle(pairs)
    return pairs


def pages(tokens, page):
    return -(-tokens // page)


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def parents_of(pairs, rnd):
    """Draft trees: node i hangs on one of the eight nodes before it or on the last cached token (-1)."""
    return [rnd.randint(max(-1, i - 8), i - 1) for _, fresh in pairs for i in range(fresh)]


def masks_of(pairs, parents):
    out, at = [], 0
    for _, fresh in pairs:
        mine = []
        for i in range(fresh):
            p = parents[at + i]
            mine.append((1 << i) | (mine[p] if p >= 0 else 0))
        out += mine
        at += fresh
    return [m - (1 << 64) if m >> 63 else m for m in out]


def new_cache(case, layers, n_pages, gen):
    """A cache as earlier steps left it: (k, v, k_scale, v_scale), every slot filled."""
    shape = (layers, n_pages, case["kv_heads"], case["page"], case["dim"])

    def one():
        x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(generator=gen)
        if case["kind"] == "f16":
            return x, None
        codes = (x * 40).clamp_(-127, 127).to(torch.int8)
        return codes, torch.empty(shape[:-1], device="cuda").uniform_(0.01, 0.05, generator=gen)

    (k, ks), (v, vs) = one(), one()
    return k, v, ks, vs


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = random.Random(seed)
    op, page = case["op"], case["page"]
    s = dict(case=case)
    if op == "append":
        tokens, kv_heads, dim = case["tokens"], case["kv_heads"], case["dim"]
        n_pages = pages(tokens, page) + 3
        s["cache"] = new_cache(case, 1, n_pages, gen)
        s["k"] = torch.randn(tokens, kv_heads * dim, generator=gen, device="cuda")
        s["v"] = torch.randn(tokens, kv_heads * dim, generator=gen, device="cuda")
        s["k"][:, ::37] *= 12.0  # outlier channels, as keys have them
        order = rnd.sample(range(n_pages), n_pages)
        off = rnd.randrange(page)  # the chunk starts inside a page
        s["slots"] = ints([order[(off + t) // page] * page + (off + t) % page for t in range(tokens)])
        return s
    pairs = lengths(case, seed)
    batch, total = len(pairs), sum(f for _, f in pairs)
    width = max(pages(c + f, page) for c, f in pairs)
    s["cached"], s["fresh"] = ints([c for c, _ in pairs]), ints([f for _, f in pairs])
    s["total"], s["max_fresh"], s["max_len"] = total, max(f for _, f in pairs), max(c + f for c, f in pairs)
    held = [pages(c if op == "plan" else c + f, page) for c, f in pairs]
    wanted = sum(pages(c + f, page) for c, f in pairs)
    n_pages = wanted + (211 if op == "plan" else 5)
    ids = rnd.sample(range(n_pages), n_pages)
    rows, at = [], 0
    for h in held:
        rows.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    s["table"], s["n_pages"] = ints(rows).view(batch, width), n_pages
    if op == "plan":
        s["free"] = ints(ids[at:])
        s["parents"] = ints(parents_of(pairs, rnd)) if case["tree"] else None
        s["starts"] = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        s["positions"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        s["masks"] = torch.zeros(total, dtype=torch.int64, device="cuda") if case["tree"] else None
        s["needed"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    if op == "accept":
        s["cache"] = new_cache(case, case["layers"], n_pages, gen)
        paths, counts = [], []
        for _, f in pairs:
            n = rnd.randint(0, min(f, 8))
            counts.append(n)
            paths.append(sorted(rnd.sample(range(f), n)) + [0] * (case["fresh"] - n))
        s["paths"], s["counts"] = ints(paths).view(batch, case["fresh"]), ints(counts)
        s["lens"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        return s
    starts = [0]
    for _, f in pairs:
        starts.append(starts[-1] + f)
    s["starts"] = ints(starts)
    s["cache"] = new_cache(case, 1, n_pages, gen)
    s["q"] = torch.randn(total, case["heads"] * case["dim"], generator=gen, device="cuda") * 1.7
    s["masks"] = ints(masks_of(pairs, parents_of(pairs, rnd)), torch.int64) if case["tree"] else None
    s["y"] = torch.zeros(total, case["heads"] * case["dim"], device="cuda")
    return s


# ----------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------------------------------------------------
def run_own(s):
    import int8_quantized_projection_gb300 as q8

    op = s["case"]["op"]
    if op == "plan":
        q8.q8_kv_plan(s["cached"], s["fresh"], s["free"], s["table"], s["case"]["page"], s["n_pages"], s["starts"],
                      s["slots"], s["positions"], s["needed"], parents=s["parents"], masks=s["masks"])
        return plan_outputs(s)
    cache = q8.KvCache(*s["cache"])
    if op == "append":
        q8.q8_kv_append(cache, 0, s["k"], s["v"], s["slots"])
        return s["cache"]
    if op == "accept":
        q8.q8_kv_accept(cache, s["table"], s["cached"], s["fresh"], s["paths"], s["counts"], s["lens"])
        return {"cache": s["cache"], "lens": s["lens"]}
    q8.q8_tree_attention(cache, 0, s["q"], s["table"], s["cached"], s["starts"], s["y"], masks=s["masks"],
                         max_fresh=s["max_fresh"], max_len=s["max_len"])
    return s["y"]


def plan_outputs(s):
    return {k: s[k] for k in ("table", "starts", "slots", "positions", "masks", "needed")}


# ----------------------------------------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------------------------------------
def plan_plain(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    cached, fresh, total = s["cached"].long(), s["fresh"].long(), s["total"]
    batch, width = table.shape
    ends = torch.cumsum(fresh, 0)
    starts = ends - fresh
    old, new = (cached + page - 1) // page, (cached + fresh + page - 1) // page
    took = torch.cumsum(new - old, 0)
    base = took - (new - old)
    # pages old..new of every row come from the free list
    i = torch.arange(width, device="cuda")[None, :]
    at = base[:, None] + i - old[:, None]
    hand = (i >= old[:, None]) & (i < new[:, None]) & (at < free.numel())
    table.copy_(torch.where(hand, free[at.clamp(0, free.numel() - 1)], table))
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    node = t - starts[b]
    pos = cached[b] + node
    got = table[b, (pos // page).clamp(max=width - 1)].long()
    s["slots"].copy_(torch.where(got >= 0, got * page + pos % page, -1))
    s["starts"].copy_(torch.cat([starts, ends[-1:]]))
    s["needed"].copy_(took[-1:])
    s["positions"].copy_(pos)
    if s["parents"] is not None:
        # ancestors: the transitive closure of "has the parent", by squaring the reachability six times
        link = torch.zeros(batch, NODES, NODES, device="cuda")
        par = s["parents"].long()
        link[b, node, par.clamp(min=0)] = (par >= 0).float()
        link += torch.eye(NODES, device="cuda")

        def square(m):
            return (m @ m).clamp(max=1.0)

        reach = square(square(square(square(square(square(link)))))) > 0
        bits = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(NODES, device="cuda")
        mask = torch.where(reach, bits, 0).sum(-1)
        s["masks"].copy_(mask[b, node])
        s["positions"].copy_(cached[b] + reach.sum(-1)[b, node] - 1)
    return plan_outputs(s)


def quantize_plain(x):
    """Rows of the last dimension -> int8 codes and one f32 scale each, with IEEE divisions."""
    amax = x.abs().amax(-1)
    d = amax / torch.full_like(amax, 127.0)
    inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
    return torch.round(x * inv[..., None]).clamp(-127, 127).to(torch.int8), d


def append_plain(s):
    case = s["case"]
    k, v, ks, vs = s["cache"]
    page, off = (s["slots"] // case["page"]).long(), (s["slots"] % case["page"]).long()
    rows = (case["tokens"], case["kv_heads"], case["dim"])

    def put(cache, scale, x):
        if scale is None:
            cache[0].transpose(1, 2)[page, off] = x.view(rows).half()
        else:
            codes, d = quantize_plain(x.view(rows))
            cache[0].transpose(1, 2)[page, off] = codes
            scale[0].transpose(1, 2)[page, off] = d

    put(k, ks, s["k"])
    put(v, vs, s["v"])
    return s["cache"]


def accept_plain(s):
    page, table = s["case"]["page"], s["table"]
    cached, fresh, count = s["cached"].long()[:, None], s["fresh"].long()[:, None], s["counts"].long()[:, None]
    j = torch.arange(s["paths"].shape[1], device="cuda")[None, :]
    move = j < count
    idle = torch.minimum(j, fresh - 1)  # past the path a slot is copied onto itself
    src, dst = cached + torch.where(move, s["paths"].long(), idle), cached + torch.where(move, j, idle)

    def slot(pos):
        last = torch.gather(table.long(), 1, (pos // page).clamp(max=table.shape[1] - 1)).clamp(min=0)
        return last.reshape(-1), (pos % page).reshape(-1)

    (sp, so), (dp, do) = slot(src), slot(dst)

    def shift(x):
        if x is not None:
            y = x.transpose(2, 3)
            y[:, dp, do] = y[:, sp, so]

    [shift(x) for x in s["cache"]]
    s["lens"].copy_(s["cached"] + s["counts"])
    return {"cache": s["cache"], "lens": s["lens"]}


def attention_plain(s):
    case = s["case"]
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    k, v, ks, vs = s["cache"]
    batch, width, group = s["table"].shape[0], s["table"].shape[1], heads // kv_heads
    cached, starts = s["cached"].long(), s["starts"].long()
    most, keys = s["max_fresh"], s["max_len"]
    ids = s["table"].long().clamp(min=0)

    def gather(c, scale):  # [batch][kv_heads][keys][dim] in 32 bits
        x = c[0][ids].float()
        if scale is not None:
            x = x * scale[0][ids][..., None]
        return x.transpose(1, 2).reshape(batch, kv_heads, width * page, dim)[:, :, :keys]

    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    node = t - starts[b]
    q = torch.zeros(batch, most, kv_heads, group, dim, device="cuda")
    q[b, node] = s["q"].view(-1, kv_heads, group, dim)
    q = q.permute(0, 2, 3, 1, 4).reshape(batch, kv_heads, group * most, dim)
    score = torch.matmul(q, gather(k, ks).transpose(-1, -2)).view(batch, kv_heads, group, most, keys) / math.sqrt(dim)
    at = torch.arange(keys, device="cuda") - cached[:, None]  # place among the fresh tokens, negative for cached ones
    if s["masks"] is not None:
        word = torch.zeros(batch, most, dtype=torch.int64, device="cuda")
        word[b, node] = s["masks"]
        seen = ((word[:, :, None] >> at.clamp(0, NODES - 1)[:, None, :]) & 1).bool() & (at < NODES)[:, None, :]
        seen = seen | (at < 0)[:, None, :]
    else:
        seen = at[:, None, :] <= torch.arange(most, device="cuda")[None, :, None]
    seen = seen & (at < (starts[1:] - starts[:-1])[:, None])[:, None, :]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    out = torch.matmul(p.view(batch, kv_heads, group * most, keys), gather(v, vs))
    out = out.view(batch, kv_heads, group, most, dim).permute(0, 3, 1, 2, 4).reshape(batch, most, heads * dim)
    s["y"].copy_(out[b, node])
    return s["y"]


def run(state):
    if own:
        return run_own(state)
    return {"plan": plan_plain, "append": append_plain, "accept": accept_plain,
            "attention": attention_plain}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------------
def work(case):
    op, page = case["op"], case["page"]
    if op == "append":
        x = case["tokens"] * case["kv_heads"] * 2
        d = case["dim"]
        return {"bytes": x * (4 * d + (2 * d if case["kind"] == "f16" else d + 4)) + 4 * case["tokens"], "flops": x * d}
    pairs = lengths(case)
    total = sum(f for _, f in pairs)
    if op == "plan":
        took = sum(pages(c + f, page) - pages(c, page) for c, f in pairs)
        return {"bytes": 12 * len(pairs) + 8 * took + total * (20 if case["tree"] else 8), "flops": total}
    row = 2 * case["kv_heads"] * (2 * case["dim"] if case["kind"] == "f16" else case["dim"] + 4)  # one token's k and v
    if op == "accept":
        moved = sum(min(f, 8) / 2 for _, f in pairs)  # the mean path
        return {"bytes": 2 * row * case["layers"] * moved + 16 * len(pairs), "flops": moved}
    flops = 0
    for c, f in pairs:
        seen = f * c + (f * (f + 1) // 2 if not case["tree"] else 4 * f)  # (row, visible key) pairs of a head
        flops += 4 * case["heads"] * case["dim"] * seen
    return {"bytes": row * sum(c + f for c, f in pairs if f) + 8 * total * case["heads"] * case["dim"], "flops": flops}


# ----------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("plan", "accept"):
        return None  # whole numbers, and values that are moved
    s = prepare(case, seed)
    page, kv_heads, dim = case["page"], case["kv_heads"], case["dim"]
    k, v, ks, vs = s["cache"]
    if case["op"] == "append":
        slots = s["slots"].tolist()
        place = torch.tensor([x // page for x in slots]).cuda(), torch.tensor([x % page for x in slots]).cuda()

        def stored(cache, scale, x):
            x = x.double().view(-1, kv_heads, dim)
            if scale is None:
                c = cache.double()
                for h in range(kv_heads):
                    c[0, place[0], h, place[1]] = x[:, h]
                return c, None
            d = scale.double()
            for h in range(kv_heads):
                d[0, place[0], h, place[1]] = x[:, h].abs().max(-1).values / 127.0
            return None, d

        (ck, dk), (cv, dv) = stored(k, ks, s["k"]), stored(v, vs, s["v"])
        return ck, cv, dk, dv
    heads = case["heads"]
    group = heads // kv_heads
    y = torch.zeros(s["total"], heads, dim, dtype=torch.float64, device="cuda")
    cached, starts, masks = s["cached"].tolist(), s["starts"].tolist(), s["masks"]
    for b, n in enumerate(cached):
        first, fresh = starts[b], starts[b + 1] - starts[b]
        if fresh == 0:
            continue
        length = n + fresh
        ids = s["table"][b, :pages(length, page)].long()
        place = torch.arange(length, device="cuda") - n
        if masks is None:
            hidden = place[None, :] > torch.arange(fresh, device="cuda")[:, None]
        else:
            word = masks[first:first + fresh]
            hidden = (place >= 0)[None, :] & (((word[:, None] >> place.clamp(0, 63)[None, :]) & 1) == 0)
        for h in range(kv_heads):
            kk = k[0, ids, h].double()
            vv = v[0, ids, h].double()
            if ks is not None:
                kk = kk * ks[0, ids, h].double()[..., None]
                vv = vv * vs[0, ids, h].double()[..., None]
            kk, vv = kk.reshape(-1, dim)[:length], vv.reshape(-1, dim)[:length]
            for a in range(h * group, (h + 1) * group):
                x = s["q"][first:first + fresh, a * dim:(a + 1) * dim].double()
                e = (x @ kk.T) * dim ** -0.5
                e[hidden] = -math.inf
                e = torch.softmax(e, dim=-1)
                y[first:first + fresh, a] = e @ vv
    return y.view(s["total"], heads * dim)
