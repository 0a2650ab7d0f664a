"""The 4-bit cache at the ends of the calls' ranges, as test_gpu_decode_limits.py does the others: lengths past the block
table, token ranges past the rows or out of order, a replayed graph on new lengths."""
import numpy as np
import pytest
import torch

import int4_util as I4
import paged_util as U
from test_gpu_decode_limits import _ints
from test_gpu_decode_ops import M, _randn

pytestmark = pytest.mark.gpu

LOST = 2.0 ** -30


def held(cache):
    return [t.clone() for t in (cache.k, cache.v, cache.ks, cache.vs)]


def full_cache(page, pages, Hkv, d, other):
    """The first sequence fills every page of its table, all of them valid; a second of `other` positions."""
    cache = I4.Cache([page * pages, other], page, Hkv, d, seed=31)
    table = cache.table[:, :pages].clone()
    spare = [x for x in range(cache.k.shape[0]) if not bool((table == x).any())]
    need = -(-other // page)
    for i in range(need, pages):
        table[1, i] = spare[(i - need) % len(spare)]
    cache.table = table
    return cache


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,over", [(1, 1), (1, 2), (4, 1), (4, 3), (4, 4), (4, 9), (32, 1), (32, 40)])
def test_append_past_the_table_leaves_cached_slots(d, n, over):
    m = M()
    page, pages, Hq, Hkv, other = 16, 4, 4, 2, 50
    cap = page * pages
    cache = full_cache(page, pages, Hkv, d, other)
    q, k, v = _randn((2 * n, Hq, d), 1), _randn((2 * n, Hkv, d), 2), _randn((2 * n, Hkv, d), 3)
    f, _ = m.mnw_rope_frequencies(d, 1e4, device="cuda")
    keep = max(0, n - over)
    want = held(cache)
    rows = torch.cat([torch.arange(keep), torch.arange(n, 2 * n)]).cuda()
    want_q = m.mnw_kv_append(q[rows], k[rows], v[rows], want[0], want[1], cache.table, _ints([cap, other]), inv_freq=f,
                             k_scale=want[2], v_scale=want[3], q_start=_ints([0, keep, keep + n]))
    err = _ints([0])
    got_q = m.mnw_kv_append(q, k, v, cache.k, cache.v, cache.table, _ints([cap + over, other]), inv_freq=f, err=err, **cache.kw())
    assert all(torch.equal(a, b) for a, b in zip(held(cache), want)) and torch.equal(got_q[rows], want_q)
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH | m.DEVERR_BAD_PAGE


def test_append_rows_past_the_last_keep_the_others_positions():
    m = M()
    n, page, pages, Hkv, d = 6, 16, 4, 2, 64
    cache = full_cache(page, pages, Hkv, d, 50)
    k, v = _randn((2 * n, Hkv, d), 2), _randn((2 * n, Hkv, d), 3)
    want = held(cache)
    m.mnw_kv_append(None, k, v, want[0], want[1], cache.table, _ints([64, 45]), k_scale=want[2], v_scale=want[3])
    err = _ints([0])
    m.mnw_kv_append(None, k, v, cache.k, cache.v, cache.table, _ints([64, 50]), q_start=_ints([0, n, 2 * n + 5]), err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    assert all(torch.equal(a, b) for a, b in zip(held(cache), want))


@pytest.mark.parametrize("n,over", [(1, 1), (4, 1), (4, 3), (4, 7), (7, 2), (32, 5), (40, 1), (40, 39)])
@pytest.mark.parametrize("blk", [1, 32])
def test_attention_past_the_table(n, over, blk):
    m = M()
    page, pages, Hq, Hkv, d, other = 16, 20, 8, 2, 128, 77
    cache = full_cache(page, pages, Hkv, d, other)
    q = _randn((2 * n, Hq, d), 1)
    err = _ints([0])
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, _ints([page * pages + over, other]), blk, 0.09, want_lse=True,
                                err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    keep = max(0, n - over)
    assert (out[keep:n] == 0).all() and (lse[keep:n] == -np.inf).all()
    rows = torch.cat([torch.arange(keep), torch.arange(n, 2 * n)]).cuda()
    U.check_attention(out[rows], lse[rows], q[rows], [keep, n], cache, blk, 0.09, lost=LOST)


@pytest.mark.parametrize("G", [1, 2, 4, 9])
def test_attention_more_tokens_than_the_table_has_positions(G):
    m = M()
    cache = I4.Cache([4], 4, 2, 128, seed=8)
    q = _randn((8, 2 * G, 128), 9)
    err = _ints([0])
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table[:, :1].contiguous(), _ints([6]), 1, 0.09, want_lse=True,
                                err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    U.check_attention(out[2:6], lse[2:6], q[2:6], [4], cache, 1, 0.09, lost=LOST)
    rest = [0, 1, 6, 7]
    assert (out[rest] == 0).all() and (lse[rest] == -np.inf).all()


@pytest.mark.parametrize("G", [2, 7, 16])
@pytest.mark.parametrize("starts", [[0, 9, 0, 9], [0, 3, 2, 9], [9, 0, 9, 9], [0, 50, -4, 9]])
def test_attention_writes_nothing_where_token_ranges_descend(G, starts):
    m = M()
    cache = I4.Cache([500, 40, 333], 16, 2, 128, seed=6)
    q = _randn((9, 2 * G, 128), 2)
    out, lse = torch.full_like(q, 7.0), torch.full((9, 2 * G), 7.0, device="cuda")
    ws = torch.full((m.mnw_attn_paged_workspace_size(3, 9, 2 * G, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    err = _ints([0])
    args = (q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.1)
    m.mnw_attn_paged(*args, q_start=_ints(starts), out=out, lse=lse, ws=ws, err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    assert (out == 7.0).all() and (lse == 7.0).all()
    m.mnw_attn_paged(*args, q_start=_ints([0, 2, 3, 9]), out=out, lse=lse, ws=ws, **cache.kw())
    U.check_attention(out, lse, q, [2, 1, 6], cache, 1, 0.1, lost=LOST)


@pytest.mark.parametrize("G", [1, 4, 12, 48])
def test_attention_graph_replayed_on_new_data(G):
    """Items shared by several runs, joined by the last arrival (up to 4 rows) or a second kernel; the workspace kept."""
    m = M()
    cache = I4.Cache([4000, 1333], 16, 4, 128, seed=3)
    q = _randn((2, 4 * G, 128), 2)
    ws = torch.full((m.mnw_attn_paged_workspace_size(2, 2, 4 * G, 4, 128),), 255, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((2, 4 * G), device="cuda")
    args = (q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.09)
    m.mnw_attn_paged(*args, out=out, lse=lse, ws=ws, **cache.kw())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            m.mnw_attn_paged(*args, out=out, lse=lse, ws=ws, **cache.kw())
    for i, now in enumerate([[4000, 1333], [900, 1], [40, 1000], [4000, 1333], [3999, 1332], [1, 1], [4000, 64]] * 4):
        cache.cache_lens.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(_randn(q.shape, 100 + i))
        cache.v.copy_(cache.v.flip(-1))
        out.fill_(3.0)
        graph.replay()
        want, want_lse = m.mnw_attn_paged(*args, want_lse=True, **cache.kw())
        assert torch.equal(out, want) and torch.equal(lse, want_lse), i
