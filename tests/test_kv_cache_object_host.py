"""KvCache: what its descriptor was made from can be read and not replaced."""
import pytest

import int8_quantized_projection_gb300 as q8p

NAMES = ("k", "v", "k_scale", "v_scale", "kv_heads", "page_size", "head_dim", "dev", "ref")


@pytest.mark.parametrize("name", NAMES)
def test_fields_are_read_only(name):
    cache = q8p.KvCache.__new__(q8p.KvCache)  # without tensors: they would have to be on a GPU
    setattr(cache, "_" + name, name)
    assert getattr(cache, name) == name
    with pytest.raises(AttributeError):
        setattr(cache, name, None)
    with pytest.raises(AttributeError):
        cache.another = 1
