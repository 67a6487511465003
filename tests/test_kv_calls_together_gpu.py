"""The cache's calls beside one another and at their edges: two attention calls in flight at once, two graphs over one
workspace, the largest batch, a batch with nothing to do, a workspace full of anything, and waits that run out."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest

from . import _kv_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Prepared:
    """A case's tensors on the device and the call over them."""

    def __init__(self, case, bound=None):
        import torch

        self.case = case
        self.cache, self.q, self.table = case.cache(), case.dev(case.q), case.dev(case.table)
        self.cached, self.starts = case.dev(np.array(case.cached, np.int32)), case.dev(case.starts)
        self.y = torch.full((case.total, case.heads * case.d), float("nan"), device="cuda")
        self.most, self.bound = max(case.fresh), bound or self.table.shape[1] * case.page
        self.ws = torch.empty(case.q8.q8_tree_attention_workspace_bytes(self.cache, case.heads, self.most),
                              dtype=torch.uint8, device="cuda")

    def run(self, stream=None, ws=None):
        self.case.q8.q8_tree_attention(self.cache, 0, self.q, self.table, self.cached, self.starts, self.y,
                                       max_fresh=self.most, max_len=self.bound,
                                       workspace=self.ws if ws is None else ws, stream=stream)

    def check(self):
        want, lim = self.case.reference()
        ref.assert_within(self.y.cpu().numpy(), want, lim)


def some(int8):
    return [Prepared(ref.Case(*c, int8), bound)
            for bound in (None, 1 << 20)  # a cluster or a CTA per unit; the line
            for c in ((90, [3000, 20], [1, 1], 28, 4, 128, 64),  # 8 rows a unit
                      (91, [2000, 900, 5], [2, 1, 2], 14, 2, 128, 32),  # 16
                      (92, [500, 0], [40, 33], 8, 1, 128, 16))]  # 128


@pytest.mark.parametrize("int8", [False, True])
def test_calls_in_flight_at_once(q8, int8):
    import torch

    calls = some(int8)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(8):
        for c, s in zip(calls, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c in calls:
        c.check()
    q8.q8_check()


@pytest.mark.parametrize("int8", [False, True])
def test_graphs_that_share_a_workspace_follow_one_another(q8, int8):
    import torch

    calls = some(int8)
    ws = max((c.ws for c in calls), key=lambda w: w.numel())
    s = torch.cuda.Stream()
    graphs = []
    for c in calls:
        c.run(ws=ws)  # sets the kernel's attributes before the capture
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            c.run(stream=s, ws=ws)
        graphs.append(g)
    for c in calls:
        c.y.fill_(float("nan"))
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for c in calls:
        c.check()
    q8.q8_check()


@pytest.mark.parametrize("int8", [False, True])
def test_the_workspace_may_hold_anything(q8, int8):
    for c in some(int8):
        c.ws.fill_(255)
        c.run()
        c.check()
    q8.q8_check()


@pytest.mark.parametrize("heads", [4, 16, 40])
def test_the_largest_batch(q8, heads):
    """4096 sequences, most of them empty or short: 8, 16 and 128 rows a unit."""
    rng = np.random.default_rng(heads)
    fresh = (rng.random(4096) < 0.3).astype(int)
    fresh[[0, 4095]] = 1
    cached = np.where(rng.random(4096) < 0.8, 0, rng.integers(0, 40, 4096))
    cached[17], fresh[17] = 3000, 1
    c = Prepared(ref.Case(93, cached.tolist(), fresh.tolist(), heads, 1, 64, 16, False))
    c.run()
    c.check()
    q8.q8_check()


def test_a_batch_past_the_largest_is_refused(q8):
    c = Prepared(ref.Case(94, [1], [1], 4, 1, 64, 16, False))
    z = c.case.torch.zeros(4097, dtype=c.case.torch.int32, device="cuda")
    with pytest.raises(q8.Q8Error):
        q8.q8_tree_attention(c.cache, 0, c.q, z[:, None].expand(-1, 2).contiguous(), z,
                             c.case.torch.zeros(4098, dtype=c.case.torch.int32, device="cuda"), c.y, max_fresh=1, max_len=8)


@pytest.mark.parametrize("heads", [4, 16, 40])
def test_nothing_fresh_writes_nothing(q8, heads):
    import torch

    c = Prepared(ref.Case(95, [40, 0, 7], [1, 1, 1], heads, 1, 64, 16, False))
    c.starts.zero_()
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.y).all()
    q8.q8_check()


_CHILD = textwrap.dedent(
    """
    import ctypes, sys
    sys.path.insert(0, ROOT)
    import numpy as np, torch
    from int8_quantized_projection_gb300 import build
    build.LIB = LIB
    import int8_quantized_projection_gb300 as q8
    from tests import _kv_ref as ref
    from tests.test_kv_calls_together_gpu import Prepared, some
    out = {}
    for int8 in (False, True):
        long = [Prepared(ref.Case(96, [60000], [n], 14, 2, 128, 64, int8), 1 << 20) for n in (1, 2, 16)]
        for n, c in enumerate(long + some(int8)):
            c.run()
            lib = q8.lib()
            st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
            out[int8, n] = lib.q8_check(st), lib.q8_check(st)
    print("RESULT", out)
    """
)


def test_waits_that_run_out_report_a_timeout(tmp_path):
    """A build whose waits give up at once: every attention kernel records the timeout, lets its copies land and returns.
    Over short contexts the copies may be there before the first wait: no report then, but never another."""
    from int8_quantized_projection_gb300 import build

    lib = build.build(extra=["-DQ8_WAIT_LIMIT_NS=0ull"], lib_path=str(tmp_path / "libq8proj_waits0.so"))
    prog = f"ROOT = {ROOT!r}\nLIB = {lib!r}\n" + _CHILD
    r = subprocess.run([sys.executable, "-c", prog], capture_output=True, text=True, timeout=180, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got = eval([ln for ln in r.stdout.splitlines() if ln.startswith("RESULT")][-1].split(" ", 1)[1])
    assert len(got) == 18 and all(v in ((5, 0), (0, 0)) for v in got.values()), got  # Q8_ERR_DEVICE_TIMEOUT, then cleared
    assert all(got[int8, n] == (5, 0) for int8 in (False, True) for n in range(3)), got
