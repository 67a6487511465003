"""A serving loop over the paged cache: plan, append, attention into the plane, o projection, accept; step after step,
eagerly, on another stream and replayed from one captured graph."""
import numpy as np
import pytest

import oracle
from int8_quantized_projection_gb300 import synthetic as syn

from . import _kv_ref as ref
from ._parity import assert_gemm_close

pytestmark = pytest.mark.gpu

HEADS, KV, D, PAGE, LAYERS, BATCH, NODES = 14, 2, 64, 16, 2, 3, 7


class Loop:
    """Drives the calls and keeps, on the host, each sequence's k and v rows as a plain list."""

    def __init__(self, q8, int8, n_out=96):
        import torch

        self.q8, self.torch, self.int8 = q8, torch, int8
        self.rng = np.random.default_rng(50 + int8)
        self.cache = q8.empty_kv_cache(LAYERS, 64, KV, PAGE, D, int8)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cap = BATCH * NODES
        self.table = torch.full((BATCH, 12), -1, dtype=torch.int32, device="cuda")
        self.cached, self.fresh, self.held, self.held_out = i32(BATCH), i32(BATCH), i32(BATCH), i32(BATCH)
        self.starts, self.slots, self.positions, self.needed = i32(BATCH + 1), i32(self.cap), i32(self.cap), i32(1)
        self.parents, self.masks = i32(self.cap), torch.zeros(self.cap, dtype=torch.int64, device="cuda")
        self.free = torch.arange(64, dtype=torch.int32, device="cuda").flip(0).contiguous()
        self.paths, self.counts, self.lens = i32(BATCH, NODES), i32(BATCH), i32(BATCH)
        z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        self.q, self.k, self.v = z(LAYERS, self.cap, HEADS * D), z(LAYERS, self.cap, KV * D), z(LAYERS, self.cap, KV * D)
        self.y = torch.full((LAYERS, self.cap, HEADS * D), float("nan"), device="cuda")
        self.plane = [q8.empty_plane(self.cap, HEADS * D) for _ in range(LAYERS)]
        for qs, ds in self.plane:
            qs.zero_(), ds.zero_()
        self.blob = syn.q8_0_weights(syn.rng(80, int(int8)), n_out, HEADS * D)[0]
        self.w, self.n_out = torch.from_numpy(self.blob).cuda(), n_out
        self.out = z(LAYERS, 16, n_out)
        nbytes = q8.q8_tree_attention_workspace_bytes(self.cache, HEADS, NODES)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.host = [[[] for _ in range(BATCH)] for _ in range(LAYERS)]  # kept (k, v) rows per layer and sequence
        self.len = [0] * BATCH

    def draw(self, most=NODES):
        r, t = self.rng, self.torch
        self.hf = [int(r.integers(0, most + 1)) for _ in range(BATCH)]
        if sum(self.hf) == 0:
            self.hf[0] = 1
        self.hp, self.hm = [], []
        for f in self.hf:
            p, m = ref.tree(r, f)
            self.hp += p
            self.hm += m
        pad = self.cap - len(self.hp)
        up = lambda a, dt=np.int32: t.from_numpy(np.asarray(a, dt)).cuda()  # noqa: E731
        self.fresh.copy_(up(self.hf)), self.cached.copy_(up(self.len))
        self.parents.copy_(up(self.hp + [0] * pad))
        for x in (self.q, self.k, self.v):
            x.copy_(t.from_numpy(r.normal(0, 1, x.shape).astype(np.float32)))
        self.paths.zero_()
        self.hc = []
        for b, f in enumerate(self.hf):
            # a path from the root through the tree
            at = sum(self.hf[:b])
            path = []
            if f:
                node = int(r.integers(0, f))
                while node >= 0:
                    path.append(node)
                    node = self.hp[at + node]
            path = path[::-1]
            self.hc.append(path)
            if path:
                self.paths[b, :len(path)] = up(path)
        self.counts.copy_(up([len(p) for p in self.hc]))

    def launch(self, stream=None):
        q8 = self.q8
        q8.q8_kv_plan(self.cached, self.fresh, self.free, self.table, PAGE, 64, self.starts, self.slots, self.positions,
                      self.needed, parents=self.parents, masks=self.masks, held=self.held, held_out=self.held_out,
                      stream=stream)
        for layer in range(LAYERS):
            qs, ds = self.plane[layer]
            q8.q8_kv_append(self.cache, layer, self.k[layer], self.v[layer], self.slots, stream=stream)
            q8.q8_tree_attention(self.cache, layer, self.q[layer], self.table, self.cached, self.starts, self.y[layer],
                                 qs=qs, ds=ds, masks=self.masks, max_fresh=NODES, max_len=12 * PAGE, workspace=self.ws,
                                 stream=stream)
            q8.q8_0_gemv_batched(self.w, self.n_out, HEADS * D, qs, ds, 16, self.out[layer], stream=stream)
        q8.q8_kv_accept(self.cache, self.table, self.cached, self.fresh, self.paths, self.counts, self.lens, stream=stream)

    def stored(self, x):
        """What the cache keeps of rows [kv][d]."""
        x = x.reshape(KV, D)
        if not self.int8:
            return x.astype(np.float16).astype(np.float64)
        d = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
        code = np.clip(np.rint(x * (np.float32(1) / d)[:, None]), -127, 127)
        return code.astype(np.float64) * d[:, None].astype(np.float64)

    def verify(self):
        total = sum(self.hf)
        self.q8.q8_check()
        assert self.starts.cpu().tolist() == np.concatenate([[0], np.cumsum(self.hf)]).tolist()
        assert self.lens.cpu().tolist() == [n + len(p) for n, p in zip(self.len, self.hc)]
        q, k, v = (x.cpu().numpy() for x in (self.q, self.k, self.v))
        for layer in range(LAYERS):
            rows = []  # a dense [batch][kv][tokens][d] cache: one page per sequence
            most = max(n + f for n, f in zip(self.len, self.hf))
            kd, vd = (np.zeros((BATCH, KV, max(most, 1), D)) for _ in range(2))
            at = 0
            for b in range(BATCH):
                mine = list(self.host[layer][b])
                new = [(self.stored(k[layer, at + i]), self.stored(v[layer, at + i])) for i in range(self.hf[b])]
                for t, (a, c) in enumerate(mine + new):
                    kd[b, :, t], vd[b, :, t] = a, c
                rows.append((mine, new))
                at += self.hf[b]
            want, lim = ref.attention(q[layer][:total], kd, vd, max(most, 1), np.arange(BATCH)[:, None], self.len, self.hf,
                                      HEADS, D ** -0.5, self.hm)
            ref.assert_within(self.y[layer][:total].cpu().numpy(), want, lim, f"layer {layer}")
            qs, ds = (p.cpu().numpy() for p in self.plane[layer])
            t16 = min(16, total)
            yr, ar = oracle.gemm(self.blob, self.n_out, HEADS * D, qs[:16], ds.view(np.uint32)[:16])
            assert_gemm_close(self.out[layer][:t16].cpu().numpy(), yr[:t16], ar[:t16], "o projection")
            for b in range(BATCH):
                mine, new = rows[b]
                self.host[layer][b] = mine + [new[i] for i in self.hc[b]]
        self.len = [n + len(p) for n, p in zip(self.len, self.hc)]
        used = int(self.needed.item())
        self.free = self.torch.cat([self.free[used:], self.free[:used]])  # the host drops what was taken
        self.held.copy_(self.held_out)


@pytest.mark.parametrize("int8", [False, True])
def test_steps(q8, int8):
    loop = Loop(q8, int8)
    for _ in range(6):
        loop.draw()
        loop.launch()
        loop.verify()


def test_steps_on_another_stream(q8):
    import torch

    loop = Loop(q8, True)
    s = torch.cuda.Stream()
    for _ in range(3):
        loop.draw()
        s.wait_stream(torch.cuda.current_stream())
        loop.launch(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        loop.verify()


def test_one_graph_replayed_for_steps_of_other_lengths(q8):
    """The lengths are device data, so the graph captured for one step serves the next ones."""
    import torch

    loop = Loop(q8, False)
    loop.draw()
    loop.launch()  # sets the kernels' attributes before the capture
    loop.verify()
    free = loop.free  # one buffer for every replay
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        loop.launch(stream=s)
    for most in (NODES, 1, 3, NODES):
        loop.draw(most)
        free.copy_(loop.free)
        loop.free = free
        g.replay()
        loop.verify()


def test_bound_calls_repeat(q8):
    import torch

    c = ref.Case(60, [40, 9], [3, 2], 4, 2, 64, 16, False)
    y = torch.zeros(5, 4 * 64, device="cuda")
    b = q8.q8_tree_attention(c.cache(), 0, c.dev(c.q), c.dev(c.table), c.dev(np.array(c.cached, np.int32)), c.dev(c.starts), y,
                             max_fresh=3, bind=True)
    b()
    want = y.clone()
    y.zero_()
    b()
    assert torch.equal(y, want)
    w, lim = c.reference()
    ref.assert_within(y.cpu().numpy(), w, lim)
