"""A value that is not finite, in the 4-bit cache, reaches the query rows that see it and no others."""
import pytest
import torch

import int4_util as I4
import paged_util as U
from test_gpu_decode_ops import M, _randn
from test_gpu_int4_hidden_keys import LOST, ROWS, positions, put, until

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hq,Hkv", ROWS)
@pytest.mark.parametrize("before,blk,page", [(0, 1, 16), (150, 1, 16), (96, 32, 20)])
def test_value_that_is_not_finite(n, Hq, Hkv, d, before, blk, page):
    m = M()
    scale = d ** -0.5
    q = _randn((n, Hq, d), n + d)
    for i, value in zip(positions(n, before, blk), (float("inf"), float("nan"), float("-inf"))):
        cache = I4.Cache([before + n], page, Hkv, d, seed=n + i)
        k, v = torch.zeros((1, Hkv, d), dtype=torch.bfloat16, device="cuda"), _randn((1, Hkv, d), 2)
        v[0, :, d // 3] = value
        put(m, cache, k, v, before + i)
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, blk, scale, want_lse=True, **cache.kw())
        hidden = max(0, (before + i) // blk * blk - before)
        assert torch.isnan(out[hidden:]).all()
        assert torch.isfinite(lse).all()  # the scores are finite
        if hidden:
            U.check_attention(out[:hidden], lse[:hidden], q[:hidden], [hidden], until(cache, before + hidden), blk, scale, lost=LOST)


@pytest.mark.parametrize("n,Hq,Hkv", [(12, 1, 1), (64, 1, 1), (200, 1, 1)])
def test_values_in_one_tile_of_several_sequences(n, Hq, Hkv):
    """The last row of one sequence; the others, and its own rows before, stay what the formula gives."""
    m = M()
    d, lens = 128, [n + 300, n + 20, n]
    for bad in range(3):
        cache = I4.Cache(lens, 16, Hkv, d, seed=bad)
        k, v = torch.zeros((1, Hkv, d), dtype=torch.bfloat16, device="cuda"), torch.full((1, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        m.mnw_kv_append(None, k, v, cache.k, cache.v, cache.table[bad:bad + 1], cache.cache_lens[bad:bad + 1], **cache.kw())
        q = _randn((3 * n, Hq, d), 5)
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.09, want_lse=True, **cache.kw())
        last = bad * n + n - 1
        assert torch.isnan(out[last]).all()
        for b in range(3):
            keep = n - (b == bad)
            part = until(cache, lens[b] - (b == bad))
            part.rows = [cache.rows[b]]
            at = slice(b * n, b * n + keep)
            U.check_attention(out[at], lse[at], q[at], [keep], part, 1, 0.09, lost=LOST)
