"""Attention over the 4-bit cache where scores are huge, over values of several magnitudes."""
import pytest
import torch

import int4_util as I4
from test_gpu_decode_ops import M, _randn
from test_gpu_int4_magnitudes import row_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq", [1, 9, 20])
@pytest.mark.parametrize("log2", [-60, -30, 0, 12, 30, 60])
def test_huge_scores_over_large_and_small_values(Hq, log2):
    """Scores of 10^31, where a score and the logarithm of a value's scale no longer add up: the largest key's value."""
    m = M()
    cache = I4.Cache([50], 16, 1, 128, seed=5, spread=0.0)
    lens = cache.cache_lens
    k = torch.from_numpy(cache.rows[0][0].numpy()).bfloat16().cuda()
    v = (_randn((50, 1, 128), 6).float() * 2.0 ** log2).bfloat16()
    m.mnw_kv_append(None, k, v, cache.k, cache.v, cache.table, lens, **cache.kw())
    pos = torch.arange(50)
    pg, sl = cache.table_host[0, pos // 16].long(), pos % 16
    keys = torch.from_numpy(I4.values(cache.k.cpu()[pg, :, sl].numpy(), cache.ks.cpu()[pg, :, sl].numpy()))[:, 0]
    for sign in (1.0, -1.0):
        q = torch.full((1, Hq, 128), sign * 2.0 ** 100, dtype=torch.bfloat16, device="cuda")
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, lens, 1, 1.0, want_lse=True, **cache.kw())
        s = sign * 2.0 ** 100 * keys.sum(1)
        best = int(s.argmax())
        want = row_of(cache, cache.v, cache.vs, best)[0]
        assert ((out[0].double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * want.abs()).all()
        assert ((lse[0].double().cpu() - s[best]).abs() <= 2.0 ** -16 * s[best].abs()).all()
