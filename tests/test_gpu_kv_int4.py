"""The 4-bit cache on the GPU against plain forms: what an append stores (bit for bit), attention over it (64 bits;
every rounding counted, see paged_util.check_attention), and its values."""
import numpy as np
import pytest
import torch

import int4_util as I4
import paged_util as U
from test_gpu_decode_ops import APPEND, ATTEND, M, _attend, _randn

pytestmark = pytest.mark.gpu

LOST = 2.0 ** -30  # products below this share of a row's largest may be lost


def _empty(cache):
    """A cache of the same pages with nothing in it."""
    c = torch.zeros_like(cache.k), torch.zeros_like(cache.v)
    s = torch.zeros_like(cache.ks), torch.zeros_like(cache.vs)
    return c + s


# ---- append ----


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"n{c[0]}-p{c[2]}-d{c[5]}-r{c[6]}{c[7][0]}")
def test_append_stores_what_the_rule_gives(case):
    """Against the rotation in FP32, operation by operation, quantised with exact integers."""
    m = M()
    counts, lens, page, Hq, Hkv, d, rot, layout, ragged = case
    cache = I4.Cache(lens, page, Hkv, d, seed=5, joint=page % 2 == 0)
    T = sum(counts)
    qkv = _randn((T, Hq + 2 * Hkv, d), 6, 2.0)
    qkv[..., 3] *= 40  # a channel far above the rest
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    f = None if rot == 0 else m.mnw_rope_frequencies(rot, 1e4, device="cuda")[0]
    start = torch.tensor(U.starts_of(counts), dtype=torch.int32, device="cuda") if ragged else None
    kw = dict(inv_freq=f, layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED, mscale=1.25, q_start=start)
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(counts, lens)])
    seq = np.repeat(np.arange(len(lens)), counts)

    def rotated(x):  # (sine and cosine as rounded from 64 bits, but for a few in 10^4, where a row may differ)
        y = x.float().cpu().numpy().copy()
        if rot:
            a = pos[:, None] * f.double().cpu().numpy()
            c, s = ((g(a).astype(np.float32) * np.float32(1.25))[:, None] for g in (np.cos, np.sin))
            i = np.arange(rot // 2)
            first, second = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            u, w = y[..., first].copy(), y[..., second].copy()
            y[..., first], y[..., second] = u * c - w * s, w * c + u * s
        return torch.from_numpy(y).bfloat16()
    before = [t.clone() for t in (cache.k, cache.v, cache.ks, cache.vs)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = m.mnw_kv_append(q, k, v, cache.k, cache.v, cache.table, cache.cache_lens, err=err, **kw, **cache.kw())
    assert int(err.item()) == 0
    differ = (got.cpu() != rotated(q)).float().mean()
    assert differ <= 2e-5  # a step of FP32 beside, in a few of 10^4, moves a BF16 value in 2^-15 of them
    pg, sl = cache.table_host[seq, pos // page].long().cuda(), torch.as_tensor(pos % page).cuda()
    for data, rec, rows in ((cache.k, cache.ks, rotated(k)), (cache.v, cache.vs, v)):
        want_data, want_rec = I4.quantise(rows.double().cpu().numpy())
        assert np.array_equal(rec[pg, :, sl].cpu().numpy(), want_rec)
        assert np.array_equal(data[pg, :, sl].cpu().numpy(), want_data)
    kept = torch.ones((cache.k.shape[0], page), dtype=torch.bool, device="cuda")
    kept[pg, sl] = False
    for now, then in zip((cache.k, cache.v, cache.ks, cache.vs), before):  # nothing else was touched
        assert torch.equal(now.transpose(1, 2)[kept], then.transpose(1, 2)[kept])


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_special_rows(d):
    """Ties, quarters of zeros, every magnitude that BF16 has, infinities and NaN (no rotation: rows go in as they are)."""
    m = M()
    g = torch.Generator().manual_seed(d)
    n = 64
    bits = torch.randint(-2 ** 15, 2 ** 15, (n, 1, d), generator=g).to(torch.int16)
    k = bits.view(torch.bfloat16).clone()
    k[~torch.isfinite(k)] = 1.0
    v = torch.randint(-14, 15, (n, 1, d), generator=g).bfloat16()  # halves of codes: 14 is two 7ths
    v[:8, :, d // 4:d // 2] = 0
    v[8:12] = 0
    v[12:20] *= 2.0 ** -110
    v[20:28, :, :d // 4] *= 2.0 ** 12
    v[28, :, 5] = float("inf")
    v[29, :, d - 1] = float("-inf")
    v[30, :, 0] = float("nan")
    v[31] = 2.0 ** 127
    cache = I4.Cache([n], 16, 1, d, seed=1)
    m.mnw_kv_append(None, k.cuda(), v.cuda(), cache.k, cache.v, cache.table, cache.cache_lens, **cache.kw())
    pos = torch.arange(n)
    pg, sl = cache.table_host[0, pos // 16].long(), pos % 16
    for data, rec, x in ((cache.k, cache.ks, k), (cache.v, cache.vs, v)):
        want_data, want_rec = I4.quantise(x.double().numpy())
        got_rec = rec.cpu()[pg, :, sl].numpy()
        s, ws = got_rec[..., :4].copy().view("<f4"), want_rec[..., :4].copy().view("<f4")
        assert np.array_equal(s, ws, equal_nan=True)
        whole = np.isfinite(ws)[..., 0]
        assert np.array_equal(got_rec[whole], want_rec[whole])
        assert np.array_equal(data.cpu()[pg, :, sl].numpy()[whole], want_data[whole])
    assert np.isnan(s[28:31]).all() and (s[8:20] == 0).all()


@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("half", 64, 48), ("interleaved", 128, 32)])
def test_append_many_tokens_as_few(layout, d, rot):
    """One call over ragged sequences with several tokens a CTA, and a call per sequence with one: the same bits."""
    m = M()
    counts, Hq, Hkv, page = [701, 1, 0, 898, 3], 6, 2, 20
    lens = [900, 1, 33, 898, 77]
    cache = I4.Cache(lens, page, Hkv, d, seed=9)
    T = sum(counts)
    q, k, v = _randn((T, Hq, d), 1), _randn((T, Hkv, d), 2), _randn((T, Hkv, d), 3)
    f, _ = m.mnw_rope_frequencies(rot, 1e4, device="cuda")
    kw = dict(inv_freq=f, layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED)
    start = U.starts_of(counts)
    few = [t.clone() for t in (cache.k, cache.v, cache.ks, cache.vs)]
    got = m.mnw_kv_append(q, k, v, cache.k, cache.v, cache.table, cache.cache_lens,
                          q_start=torch.tensor(start, dtype=torch.int32, device="cuda"), **kw, **cache.kw())
    for b, n in enumerate(counts):
        if n:
            at = slice(start[b], start[b + 1])
            one = m.mnw_kv_append(q[at], k[at], v[at], few[0], few[1], cache.table[b:b + 1], cache.cache_lens[b:b + 1],
                                  k_scale=few[2], v_scale=few[3], **kw)
            assert torch.equal(got[at], one)
    assert all(torch.equal(a, b) for a, b in zip((cache.k, cache.v, cache.ks, cache.vs), few))


def test_append_leaves_out_what_does_not_fit():
    m = M()
    cache = I4.Cache([40, 6], 16, 2, 128, seed=1)
    q, k, v = _randn((4, 4, 128), 1), _randn((4, 2, 128), 2), _randn((4, 2, 128), 3)
    f, _ = m.mnw_rope_frequencies(128, 1e4, device="cuda")
    for lens, table, code in (([40, 1], cache.table, m.DEVERR_BAD_LENGTH),  # fewer positions than new tokens
                              ([-3, 6], cache.table, m.DEVERR_BAD_LENGTH),
                              ([10 ** 6, 6], cache.table, m.DEVERR_BAD_LENGTH | m.DEVERR_BAD_PAGE),
                              ([40, 6], torch.full_like(cache.table, 1000), m.DEVERR_BAD_PAGE),
                              ([40, 6], torch.full_like(cache.table, -1), m.DEVERR_BAD_PAGE)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kc, vc, ks, vs = _empty(cache)
        m.mnw_kv_append(q, k, v, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), inv_freq=f, err=err,
                        k_scale=ks, v_scale=vs)
        assert m.mnw_moe_read_error(err) & code == code
        written = int((ks != 0).any(-1).any(1).sum())
        assert written <= (3 if code & m.DEVERR_BAD_LENGTH else 0)
        assert torch.equal((ks != 0).any(-1), (kc != 0).any(-1))


# ---- attention ----


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"n{c[0]}-L{c[1]}-p{c[2]}-d{c[5]}")
def test_attention_matches_plain(case):
    counts, lens, page, Hq, Hkv, d, blk, ragged = case
    cache = I4.Cache(lens, page, Hkv, d, seed=7, joint=page == 20)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, out, lse, scale = _attend(cache, counts, Hq, blk, ragged, err=err)
    assert int(err.item()) == 0
    U.check_attention(out, lse, q, counts, cache, blk, scale, lost=LOST)


@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 1), (7, 1, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1), (17, 1, 1), (32, 1, 1), (33, 1, 1),
                                      (4, 2, 9), (8, 2, 16), (5, 5, 31)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_rows_around_the_tiles(Hq, Hkv, n, d):
    """Query rows of a kv head at, below and above each row tile."""
    lens = [n + 300, n, n + 127, n + 1000]
    cache = I4.Cache(lens, 16, Hkv, d, seed=Hq + n)
    q, out, lse, scale = _attend(cache, [n] * 4, Hq, 4, False)
    U.check_attention(out, lse, q, [n] * 4, cache, 4, scale, lost=LOST)


def test_attention_long_split_and_many_sequences():
    cache = I4.Cache([40003], 64, 2, 128, seed=8)
    q, out, lse, scale = _attend(cache, [1], 8, 1, False)
    U.check_attention(out, lse, q, [1], cache, 1, scale, lost=LOST)
    lens = [1 + 7 * i % 90 for i in range(200)]
    cache = I4.Cache(lens, 16, 1, 64, seed=9)
    q, out, lse, scale = _attend(cache, [1] * 200, 4, 1, False)
    U.check_attention(out, lse, q, [1] * 200, cache, 1, scale, lost=LOST)


def test_attention_of_wide_scores_and_spread_values():
    """Scores over hundreds, rising along the cache, values from 2^-20 to 2^20 of each other."""
    for d, Hq in ((128, 4), (64, 32)):
        cache = I4.Cache([700], 16, 1, d, seed=3, spread=6.0)
        q = _randn((1, Hq, d), 4, 30.0)
        out, lse = M().mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, d ** -0.5, want_lse=True, **cache.kw())
        U.check_attention(out, lse, q, [1], cache, 1, d ** -0.5, lost=LOST)


def test_attention_of_huge_scores():
    """Scores of 10^31 in both directions: the largest key's value alone, and finite statistics."""
    m = M()
    cache = I4.Cache([50], 16, 1, 128, seed=5, spread=0.0)
    for Hq in (4, 40):
        for sign in (1.0, -1.0):
            q = torch.full((1, Hq, 128), sign * 2.0 ** 100, dtype=torch.bfloat16, device="cuda")
            out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 1.0, want_lse=True, **cache.kw())
            s = sign * 2.0 ** 100 * cache.rows[0][0][:, 0].sum(1)
            best = int(s.argmax())
            want = cache.rows[0][1][best, 0]
            assert ((out[0].double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * want.abs()).all()
            assert ((lse[0].double().cpu() - s[best]).abs() <= 2.0 ** -16 * s[best].abs()).all()


def test_attention_of_zero_queries_zero_rows_and_empty_sequences():
    m = M()
    cache = I4.Cache([70, 3], 16, 2, 128, seed=2)
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.1, want_lse=True, **cache.kw())
    U.check_attention(out, lse, q, [1, 1], cache, 1, 0.1, lost=LOST)
    # a cache of zeros: the mean of zeros, lse the count's logarithm
    kc, vc, ks, vs = _empty(cache)
    out, lse = m.mnw_attn_paged(_randn((2, 4, 128), 1), kc, vc, cache.table, cache.cache_lens, 1, 0.1, k_scale=ks, v_scale=vs, want_lse=True)
    assert (out == 0).all()
    want = torch.log(torch.tensor([70.0, 3.0])).cuda()[:, None].expand(2, 4)
    assert ((lse - want).abs() <= 2.0 ** -20).all()
    # lengths of zero: nothing is seen
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = m.mnw_attn_paged(_randn((2, 4, 128), 1), cache.k, cache.v, cache.table, none, 1, 0.1, want_lse=True, err=err, **cache.kw())
    assert (out == 0).all() and (lse == -float("inf")).all() and int(err.item()) == m.DEVERR_BAD_LENGTH


def test_a_row_that_is_not_finite_reaches_those_that_see_it():
    m = M()
    cache = I4.Cache([40, 40], 16, 1, 128, seed=6)
    k, v = _randn((2, 1, 128), 1), _randn((2, 1, 128), 2)
    v[1, 0, 7] = float("inf")
    m.mnw_kv_append(None, k, v, cache.k, cache.v, cache.table, cache.cache_lens, **cache.kw())
    out = m.mnw_attn_paged(_randn((2, 2, 128), 3), cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.1, **cache.kw())
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()


def test_bad_pages_read_as_zeros_and_are_reported():
    m = M()
    for Hq in (4, 40):
        cache = I4.Cache([100, 260], 16, 1, 128, seed=4)
        table = cache.table.clone()
        table[0, 2], table[1, 5] = 10 ** 6, -1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = _randn((2, Hq, 128), 5)
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, table, cache.cache_lens, 1, 0.1, want_lse=True, err=err, **cache.kw())
        assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_PAGE
        for b, page in ((0, 2), (1, 5)):
            for x in cache.rows[b]:
                x[16 * page:16 * page + 16] = 0
        U.check_attention(out, lse, q, [1, 1], cache, 1, 0.1, lost=LOST)


@pytest.mark.parametrize("page", [1, 3, 8, 100, 128, 256])
def test_pages_below_at_and_above_a_tile(page):
    for n, Hq in ((1, 4), (32, 4)):
        lens = [n + 5, n + 250, n + 513]
        cache = I4.Cache(lens, page, 1, 128, seed=page, joint=page == 8)
        q, out, lse, scale = _attend(cache, [n] * 3, Hq, 32, False)
        U.check_attention(out, lse, q, [n] * 3, cache, 32, scale, lost=LOST)


def test_pages_past_32_bit_offsets():
    """Append and attention over pages whose bytes lie past 2^32 of the cache's start (two layers in one allocation)."""
    m = M()
    Hkv, page, d = 8, 64, 128
    row = Hkv * page * d // 2  # bytes of a page
    n_pages, apart = 6, 1 << 30
    pool = torch.zeros(apart * n_pages + row, dtype=torch.uint8, device="cuda")
    kc = pool[:apart * n_pages].view(n_pages, apart)[:, :row].view(n_pages, Hkv, page, d // 2)
    vc = pool[row:apart * n_pages + row].view(n_pages, apart)[:, :row].view(n_pages, Hkv, page, d // 2)
    ks, vs = (torch.zeros((n_pages, Hkv, page, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.tensor([[5, 0, 4]], dtype=torch.int32, device="cuda")
    L = 150
    k, v = _randn((L, Hkv, d), 1), _randn((L, Hkv, d), 2)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    m.mnw_kv_append(None, k, v, kc, vc, table, lens, k_scale=ks, v_scale=vs)
    small = [torch.zeros((n_pages, Hkv, page, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    m.mnw_kv_append(None, k, v, small[0], small[1], table, lens, k_scale=ks.clone(), v_scale=vs.clone())
    assert torch.equal(kc, small[0]) and torch.equal(vc, small[1])
    for n in (1, 32):
        q = _randn((n, 16, d), 3)
        a = m.mnw_attn_paged(q, kc, vc, table, lens, 32, 0.1, k_scale=ks, v_scale=vs)
        b = m.mnw_attn_paged(q, small[0], small[1], table, lens, 32, 0.1, k_scale=ks, v_scale=vs)
        assert torch.equal(a, b)
    assert torch.equal(m.mnw_kv_values(kc, ks), m.mnw_kv_values(small[0], ks))


# ---- values ----


@pytest.mark.parametrize("d,page,Hkv,joint", [(128, 16, 2, False), (64, 5, 3, False), (128, 1, 1, True), (64, 100, 2, True)])
def test_values(d, page, Hkv, joint):
    m = M()
    cache = I4.Cache([300, 7], page, Hkv, d, seed=2, joint=joint)
    for data, rec in ((cache.k, cache.ks), (cache.v, cache.vs)):
        got = m.mnw_kv_values(data, rec)
        codes = torch.from_numpy(I4.unpack(data.cpu().numpy())).float()
        r = rec.cpu()
        f = r[..., :4].contiguous().view(torch.float32) * r[..., 4:].float()
        want = (codes.unflatten(-1, (4, -1)) * f[..., None]).flatten(-2).bfloat16()
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=-7.5), torch.nan_to_num(want, nan=-7.5))
    int8 = U.Cache([300, 7], page, Hkv, d, "int8", seed=2, joint=joint and d * page % 16 == 0)
    got = m.mnw_kv_values(int8.v, int8.vs)
    want = (int8.v.float() * int8.vs[..., None]).bfloat16()
    assert torch.equal(torch.nan_to_num(got, nan=-7.5), torch.nan_to_num(want, nan=-7.5))


def test_values_of_more_chunks_than_31_bits():
    m = M()
    Hkv, page, d = 8, 256, 128
    n_pages = (1 << 31) // (Hkv * page * (d // 8)) + 3
    cache = torch.zeros((n_pages, Hkv, page, d // 2), dtype=torch.uint8, device="cuda")
    rec = torch.zeros((n_pages, Hkv, page, 8), dtype=torch.uint8, device="cuda")
    small = I4.Cache([3 * page], page, Hkv, d, seed=3, spread=0.0)
    far = torch.tensor([0, n_pages // 2, n_pages - 1], device="cuda")
    own = small.table[0, :3].long()
    cache[far], rec[far] = small.k[own], small.ks[own]
    got = m.mnw_kv_values(cache, rec)
    assert torch.equal(got[far], m.mnw_kv_values(small.k[own], small.ks[own]))
    assert (got[1] == 0).all() and (got[n_pages - 2] == 0).all()


# ---- together ----


@pytest.mark.parametrize("d,n,Hq,Hkv", [(128, 1, 8, 2), (64, 32, 8, 2)])
def test_append_and_attention_in_a_replayed_graph(d, n, Hq, Hkv):
    """Captured once; new tokens, lengths and pages are read from the device at each replay."""
    m = M()
    B, page, most = 3, 16, 24
    kc, vc = (torch.zeros((B * most, Hkv, page, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((B * most, Hkv, page, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    kw = dict(k_scale=ks, v_scale=vs)
    table = torch.arange(B * most, dtype=torch.int32, device="cuda").view(B, most).flip(1).contiguous()
    lens = torch.tensor([n, 2 * n + 40, 130 + n], dtype=torch.int32, device="cuda")
    qkv = _randn((B * n, Hq + 2 * Hkv, d), 1)
    f, _ = m.mnw_rope_frequencies(d, 1e4, device="cuda")

    def step():
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        q = m.mnw_kv_append(q, k, v, kc, vc, table, lens, f, **kw)
        return m.mnw_attn_paged(q, kc, vc, table, lens, 32, d ** -0.5, **kw)
    start = lens.clone()
    past = [_randn((B * 130, Hkv, d), s) for s in (2, 3)]
    m.mnw_kv_append(None, past[0], past[1], kc, vc, table, torch.full_like(lens, 130), f, **kw)
    saved = [t.clone() for t in (kc, vc, ks, vs)]
    want = []
    for i in range(4):
        qkv.copy_(_randn(tuple(qkv.shape), 10 + i))
        lens.copy_(start + i * n)
        want.append(step().clone())
    for t, s in zip((kc, vc, ks, vs), saved):
        t.copy_(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lens.copy_(start)
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t, s in zip((kc, vc, ks, vs), saved):
        t.copy_(s)
    for i in range(4):
        qkv.copy_(_randn(tuple(qkv.shape), 10 + i))
        lens.copy_(start + i * n)
        graph.replay()
        assert torch.equal(out, want[i]), i


@pytest.mark.parametrize("at", [1000, 131071, 16777217, 1 << 30])
def test_rotation_keeps_far_positions(at):
    """Angles at far positions, by a table that sends every page to page 0; negative frequencies turn the other way."""
    m = M()
    page = 65536
    table = torch.zeros((1, at // page + 1), dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((1, 1, page, 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((1, 1, page, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    q, kv = _randn((3, 2, 64), 1), _randn((3, 1, 64), 2)
    f, _ = m.mnw_rope_frequencies(64, 1e4, device="cuda")
    f[5] *= -1
    lens = torch.tensor([at], dtype=torch.int32, device="cuda")
    for layout in ("half", "interleaved"):
        got = m.mnw_kv_append(q, kv, kv, kc, vc, table, lens, inv_freq=f, k_scale=ks, v_scale=vs,
                              layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED)
        ref, size = U.rotate_plain(q, np.arange(at - 3, at), f, 64, layout, 1.0)
        # BF16's half step; sine and cosine (half a step of FP32), three roundings, and 2^-64 turns a position
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -22 + at * 2.0 ** -61) * size
        assert ((got.double().cpu() - ref).abs() <= tol).all()
