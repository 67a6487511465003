"""Cases of the norm-wise tests: every kernel and both ways of sharing the units, 64 and 128 values a head."""
from . import _kv_ref as ref

# heads, key/value heads, head_dim, page; whether the fresh tokens are a tree
CASES = dict(
    rows8_d128=dict(cached=[700, 300], fresh=[1, 1], heads=28, kv_heads=4, d=128, page=16),
    rows8_d64=dict(cached=[900, 5, 400], fresh=[2, 1, 2], heads=12, kv_heads=3, d=64, page=48),
    rows16_d128=dict(cached=[700, 300], fresh=[2, 2], heads=28, kv_heads=4, d=128, page=32, tree=True),
    rows16_d64=dict(cached=[1300], fresh=[1], heads=24, kv_heads=2, d=64, page=16),
    tiles_d128=dict(cached=[600, 100], fresh=[16, 9], heads=14, kv_heads=2, d=128, page=64, tree=True),
    tiles_d64=dict(cached=[800], fresh=[64], heads=4, kv_heads=1, d=64, page=16, tree=True),
    prompt_d128=dict(cached=[130], fresh=[260], heads=7, kv_heads=1, d=128, page=32),
    long_rows8=dict(cached=[30000], fresh=[1], heads=14, kv_heads=2, d=128, page=64),
    long_tiles=dict(cached=[20000], fresh=[5], heads=16, kv_heads=2, d=128, page=64, tree=True),
)


def build(name, int8, seed=200):
    c = dict(CASES[name])
    tree = c.pop("tree", False)
    case = ref.Case(seed, int8=int8, **c)
    masks = sum((ref.tree(case.rng, f)[1] for f in case.fresh), []) if tree else None
    return case, masks
