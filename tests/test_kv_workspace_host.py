"""The workspace size that q8_tree_attention remembers: a refused call leaves nothing behind for the next one."""
import ctypes

import pytest

import int8_quantized_projection_gb300 as q8p
from int8_quantized_projection_gb300 import _binding, build

from .test_kv_abi_host import LONG, desc


class Described:
    """What the size depends on of a KvCache, without tensors."""

    def __init__(self, **kw):
        self.desc = desc(**kw)
        self._ref = ctypes.addressof(self.desc)
        self._kv_heads, self._head_dim = self.desc.kv_heads, self.desc.head_dim


@pytest.fixture(autouse=True)
def built(monkeypatch):
    build.build()
    monkeypatch.setattr(_binding, "_workspace_sizes", {})


@pytest.mark.parametrize("bad", [dict(page=8), dict(page=24), dict(layers=0), dict(n_pages=0), dict(dtype=3)])
@pytest.mark.parametrize("heads,fresh", [(28, 1), (28, 2), (28, 16)])
def test_a_refused_descriptor_leaves_no_size(bad, heads, fresh):
    assert _binding._workspace_size(Described(**bad), heads, 2, fresh, LONG) == 0
    good = Described()
    want = q8p.q8_tree_attention_workspace_bytes(good, heads, fresh)
    assert want > 0
    for _ in range(2):  # asked, then remembered
        assert _binding._workspace_size(good, heads, 2, fresh, LONG) == want


def test_sizes_that_need_none_are_remembered():
    for _ in range(2):
        assert _binding._workspace_size(Described(), 28, 2, 1, 300) == 0
    assert list(_binding._workspace_sizes.values()) == [0]


def test_refused_sizes_leave_none():
    assert _binding._workspace_size(Described(), 30, 2, 1, LONG) == 0  # 30 heads on 4
    assert not _binding._workspace_sizes
