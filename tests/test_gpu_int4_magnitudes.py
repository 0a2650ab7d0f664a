"""Attention over the 4-bit cache where values are very large or very small."""
import numpy as np
import pytest
import torch

import int4_util as I4
from test_gpu_decode_ops import M, _randn

pytestmark = pytest.mark.gpu


def row_of(cache, data, rec, at):
    """[Hkv, d] that the first sequence's cached row stands for."""
    page, slot = int(cache.table_host[0, at // cache.page]), at % cache.page
    return torch.from_numpy(I4.values(data[page, :, slot].cpu().numpy(), rec[page, :, slot].cpu().numpy()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [1, 9, 20, 40])
@pytest.mark.parametrize("log2,L", [(126, 50), (126, 30000), (121, 3000), (-99, 50), (-99, 3000)])
def test_one_key_that_counts_with_values_at_the_ends_of_the_range(d, Hq, log2, L):
    """One key's score lies hundreds above the rest, so the output is its value row: the probability's product in FP16
    (2^-11), the output in BF16 (2^-8)."""
    m = M()
    cache = I4.Cache([L], 16, 1, d, seed=d, spread=0.0)
    at = L // 3
    k = torch.full((1, 1, d), 100.0, dtype=torch.bfloat16, device="cuda")
    v = (_randn((1, 1, d), 3).float().clamp(-1.9, 1.9) * 2.0 ** log2).bfloat16()
    m.mnw_kv_append(None, k, v, cache.k, cache.v, cache.table, torch.tensor([at + 1], dtype=torch.int32, device="cuda"), **cache.kw())
    want = row_of(cache, cache.v, cache.vs, at)[0]
    q = torch.full((1, Hq, d), 4.0, dtype=torch.bfloat16, device="cuda")
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 1.0, want_lse=True, **cache.kw())
    score = 4.0 * float(row_of(cache, cache.k, cache.ks, at).sum())
    rest = 4.0 * cache.rows[0][0][:, 0].sum(1)
    rest[at] = -np.inf
    assert float(rest.max()) < score - 200  # what the case is about
    assert ((out[0].double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * want.abs()).all()
    assert ((lse[0].double().cpu() - score).abs() <= 2.0 ** -18 * score).all()
