"""A key that is not finite, in the 4-bit cache, reaches the query rows that see it and no others, whichever kernel the
number of rows leads to.  Those others are checked against the plain form, every rounding counted (paged_util)."""
import pytest
import torch

import int4_util as I4
import paged_util as U
from test_gpu_decode_ops import M, _randn

pytestmark = pytest.mark.gpu

LOST = 2.0 ** -30
ROWS = [(3, 1, 1), (12, 1, 1), (30, 1, 1), (8, 8, 2), (33, 1, 1), (64, 1, 1), (200, 1, 1), (40, 4, 2), (129, 2, 1)]  # tokens, query, kv heads


def put(m, cache, k, v, at):
    """Keys and values of position `at` into the cache (no rotation)."""
    lens = torch.tensor([at + 1], dtype=torch.int32, device="cuda")
    m.mnw_kv_append(None, k, v, cache.k, cache.v, cache.table, lens, **cache.kw())


def until(cache, length):
    """The cache's first positions as a cache of its own."""
    part = U.Cache.__new__(U.Cache)
    part.__dict__.update(cache.__dict__)
    part.lens, part.rows = [length], cache.rows
    return part


def positions(n, before, blk):
    """Token of the chunk: first, a middle one at a block's beginning, last."""
    mid = max((before + n // 2) // blk * blk - before, 0)
    return sorted({0, mid, n - 1})


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hq,Hkv", ROWS)
@pytest.mark.parametrize("before,blk,page", [(0, 1, 16), (150, 1, 16), (96, 32, 20)])
def test_key_that_is_not_finite(n, Hq, Hkv, d, before, blk, page):
    m = M()
    L = before + n
    scale = d ** -0.5
    q = _randn((n, Hq, d), n + d)
    for i, value in zip(positions(n, before, blk), (float("inf"), float("nan"), float("-inf"))):
        cache = I4.Cache([L], page, Hkv, d, seed=n + i)
        k, v = _randn((1, Hkv, d), 1), _randn((1, Hkv, d), 2)
        k[0, :, d // 3] = value
        put(m, cache, k, v, before + i)
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, blk, scale, want_lse=True, **cache.kw())
        hidden = max(0, (before + i) // blk * blk - before)  # tokens whose blocks end before that key
        assert torch.isnan(out[hidden:]).all() and torch.isnan(lse[hidden:]).all()
        if hidden:
            U.check_attention(out[:hidden], lse[:hidden], q[:hidden], [hidden], until(cache, before + hidden), blk, scale, lost=LOST)


@pytest.mark.parametrize("n,Hq,Hkv", [(12, 1, 1), (30, 1, 1), (64, 1, 1), (200, 1, 1)])
def test_infinite_key_of_an_int8_cache(n, Hq, Hkv):
    m = M()
    d, before = 128, 150
    q = _randn((n, Hq, d), n)
    for i in positions(n, before, 1):
        cache = U.Cache([before + n], 16, Hkv, d, "int8", seed=n + i)
        k, v = _randn((1, Hkv, d), 1), _randn((1, Hkv, d), 2)
        k[0, :, 7] = float("inf")
        put(m, cache, k, v, before + i)
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.09, want_lse=True, **cache.kw())
        if i:
            U.check_attention(out[:i], lse[:i], q[:i], [i], until(cache, before + i), 1, 0.09, lost=2.0 ** -38)
