"""The decode step's operators at the ends of their ranges: lengths past the
block table, token ranges past the rows."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_util as U

pytestmark = pytest.mark.gpu


def M():
    import quantized_moe_expert_routed_gb300 as m
    return m


def _randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16().cuda()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bits(cache_tensors):
    return [t.view(torch.int8 if t.dtype is torch.int8 else torch.int32 if t.dtype is torch.float32 else torch.int16)
            for t in cache_tensors if t is not None]


# ---- lengths past the table: the tokens that have no slot are left out, the others stay where they belong ----


def _full_cache(fmt, page, pages, Hkv, d, other):
    """A cache whose first sequence fills every page of its table, all of them valid, and a second of `other` positions."""
    cache = U.Cache([page * pages, other], page, Hkv, d, fmt, seed=31, stale=0.0)
    table = cache.table[:, :pages].clone()
    spare = [x for x in range(cache.k.shape[0]) if not bool((table == x).any())]
    need = -(-other // page)
    for i in range(need, pages):  # valid pages in the rest of the second row, too
        table[1, i] = spare[(i - need) % len(spare)]
    cache.table = table
    return cache


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n,over", [(1, 1), (1, 2), (4, 1), (4, 3), (4, 4), (4, 9), (32, 1), (32, 40)])
def test_append_past_the_table_leaves_cached_slots(fmt, n, over):
    m = M()
    page, pages, Hq, Hkv, d, other = 16, 4, 4, 2, 128, 50
    cap = page * pages
    cache = _full_cache(fmt, page, pages, Hkv, d, other)
    q, k, v = _randn((2 * n, Hq, d), 1), _randn((2 * n, Hkv, d), 2), _randn((2 * n, Hkv, d), 3)
    f, _ = m.mnw_rope_frequencies(d, 1e4, device="cuda")
    keep = max(0, n - over)  # tokens of the first sequence that have a slot
    want = [None if t is None else t.clone() for t in (cache.k, cache.v, cache.ks, cache.vs)]
    rows = torch.cat([torch.arange(keep), torch.arange(n, 2 * n)]).cuda()
    want_q = m.mnw_kv_append(q[rows], k[rows], v[rows], want[0], want[1], cache.table, _ints([cap, other]), inv_freq=f,
                             k_scale=want[2], v_scale=want[3], q_start=_ints([0, keep, keep + n]))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got_q = m.mnw_kv_append(q, k, v, cache.k, cache.v, cache.table, _ints([cap + over, other]), inv_freq=f, err=err,
                            **cache.kw())
    for a, b in zip(_bits((cache.k, cache.v, cache.ks, cache.vs)), _bits(want)):
        assert torch.equal(a, b)
    assert torch.equal(got_q[rows], want_q)
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH | m.DEVERR_BAD_PAGE


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_append_rows_past_the_last_keep_the_others_positions(fmt):
    """The second sequence claims 5 rows more than there are: the rows that exist are its first ones."""
    m = M()
    n, page, pages, Hkv, d = 6, 16, 4, 2, 64
    cache = _full_cache(fmt, page, pages, Hkv, d, 50)
    k, v = _randn((2 * n, Hkv, d), 2), _randn((2 * n, Hkv, d), 3)
    want = [None if t is None else t.clone() for t in (cache.k, cache.v, cache.ks, cache.vs)]
    m.mnw_kv_append(None, k, v, want[0], want[1], cache.table, _ints([64, 45]), k_scale=want[2], v_scale=want[3])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.mnw_kv_append(None, k, v, cache.k, cache.v, cache.table, _ints([64, 50]), q_start=_ints([0, n, 2 * n + 5]), err=err,
                    **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    for a, b in zip(_bits((cache.k, cache.v, cache.ks, cache.vs)), _bits(want)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n,over", [(1, 1), (4, 1), (4, 3), (4, 7), (7, 2), (32, 5), (40, 1), (40, 39)])
@pytest.mark.parametrize("blk", [1, 32])
def test_attention_past_the_table(fmt, n, over, blk):
    """Tokens past the table see nothing, the others what they saw; one to two row tiles of each kernel."""
    m = M()
    page, pages, Hq, Hkv, d, other = 16, 20, 8, 2, 128, 77
    cap = page * pages
    cache = _full_cache(fmt, page, pages, Hkv, d, other)
    q = _randn((2 * n, Hq, d), 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, _ints([cap + over, other]), blk, 0.09, want_lse=True,
                                err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    keep = max(0, n - over)
    assert (out[keep:n] == 0).all() and (lse[keep:n] == -np.inf).all()
    rows = torch.cat([torch.arange(keep), torch.arange(n, 2 * n)]).cuda()
    U.check_attention(out[rows], lse[rows], q[rows], [keep, n], cache, blk, 0.09, lost=2.0 ** -38 if fmt == "int8" else 0.0)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("G", [1, 2, 4, 9])
def test_attention_more_tokens_than_the_table_has_positions(fmt, G):
    """One tile of query rows from before the first position to past the table: the ones between see what is there."""
    m = M()
    cache = U.Cache([4], 4, 2, 128, fmt, seed=8)
    q = _randn((8, 2 * G, 128), 9)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table[:, :1].contiguous(), _ints([6]), 1, 0.09, want_lse=True,
                                err=err, **cache.kw())  # positions -2 .. 5 over 4 slots
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    U.check_attention(out[2:6], lse[2:6], q[2:6], [4], cache, 1, 0.09, lost=2.0 ** -38 if fmt == "int8" else 0.0)
    rest = [0, 1, 6, 7]
    assert (out[rest] == 0).all() and (lse[rest] == -np.inf).all()


# ---- tiles that come row by row and tiles that come whole, in turn ----


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("short", [3, 5])
def test_attention_short_and_whole_tiles_in_turn(fmt, d, short):
    """Sequences of one partly filled tile (copied row by row) in groups of `short`, each group before one of whole tiles,
    enough of them that a CTA's run takes several: the two ways of copying follow each other in the same buffers."""
    page, Hq, Hkv, n, groups = 16, 16, 4, 12, 90
    lens = []
    for i in range(groups):
        lens += [65 + (29 * i + 17 * j) % 63 for j in range(short)] + [128 * (1 + i % 5)]
    counts = [n] * len(lens)
    cache = U.Cache(lens, page, Hkv, d, fmt, seed=short)
    q = _randn((n * len(lens), Hq, d), 5)
    m = M()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 4, d ** -0.5, want_lse=True,
                                    err=err, **cache.kw())
    out, lse = call()
    for _ in range(20):  # the same bits, whatever the warps' order
        again, lse2 = call()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    assert m.mnw_moe_read_error(err) == 0
    some = list(range(0, len(lens), 7)) + [len(lens) - 1]
    pick = torch.cat([torch.arange(n * b, n * b + n) for b in some]).cuda()
    part = U.Cache.__new__(U.Cache)
    part.__dict__.update(cache.__dict__)
    part.lens, part.rows = [lens[b] for b in some], [cache.rows[b] for b in some]
    U.check_attention(out[pick], lse[pick], q[pick], [n] * len(some), part, 4, d ** -0.5,
                      lost=2.0 ** -38 if fmt == "int8" else 0.0)


# ---- token ranges out of order ----


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("G", [2, 16])
@pytest.mark.parametrize("starts", [[0, 9, 0, 9], [0, 3, 2, 9], [9, 0, 9, 9], [0, 50, -4, 9]])
def test_attention_writes_nothing_where_token_ranges_descend(fmt, G, starts):
    """Rows that several sequences claim: the outputs keep what they held, and the next call is not disturbed."""
    m = M()
    cache = U.Cache([500, 40, 333], 16, 2, 128, fmt, seed=6)
    q = _randn((9, 2 * G, 128), 2)
    out = torch.full_like(q, 7.0)
    lse = torch.full((9, 2 * G), 7.0, device="cuda")
    ws = torch.full((m.mnw_attn_paged_workspace_size(3, 9, 2 * G, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.1)
    m.mnw_attn_paged(*args, q_start=_ints(starts), out=out, lse=lse, ws=ws, err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH
    assert (out == 7.0).all() and (lse == 7.0).all()
    m.mnw_attn_paged(*args, q_start=_ints([0, 2, 3, 9]), out=out, lse=lse, ws=ws, **cache.kw())
    U.check_attention(out, lse, q, [2, 1, 6], cache, 1, 0.1, lost=2.0 ** -38 if fmt == "int8" else 0.0)


# ---- the fused join: a replayed graph brings the same call number again ----


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("G", [1, 4])
def test_attention_graph_replayed_on_new_data(fmt, G):
    """At most 4 query rows a kv head, items shared by several runs, the workspace kept between replays: each replay
    gives the bits of an eager call on another workspace."""
    m = M()
    lens = [4000, 1333]
    cache = U.Cache(lens, 16, 4, 128, fmt, seed=3)
    q = _randn((2, 4 * G, 128), 2)
    size = m.mnw_attn_paged_workspace_size(2, 2, 4 * G, 4, 128)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((2, 4 * G), device="cuda")
    args = (q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.09)
    m.mnw_attn_paged(*args, out=out, lse=lse, ws=ws, **cache.kw())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):  # two nodes share a workspace, one after the other
            m.mnw_attn_paged(*args, out=out, lse=lse, ws=ws, **cache.kw())
    for i, now in enumerate([[4000, 1333], [900, 1], [40, 1000], [4000, 1333], [3999, 1332], [1, 1], [4000, 64]] * 4):
        cache.cache_lens.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(_randn(q.shape, 100 + i))
        cache.v.copy_(cache.v.flip(-1))
        out.fill_(3.0)
        graph.replay()
        want, want_lse = m.mnw_attn_paged(*args, want_lse=True, **cache.kw())
        assert torch.equal(out, want) and torch.equal(lse, want_lse), i


# ---- angles of far positions ----

INV_2PI = Fraction(15915494309189533576888376337251436203445964574046, 10 ** 50)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("low,high", [(0, 1 << 16), (1 << 16, 10 ** 7), (10 ** 7, 1 << 27), (1 << 27, 1 << 30),
                                      (1 << 30, (1 << 31) - 131072)])
def test_rotation_angle_error(low, high, layout):
    """Positions whose angle lies next to a border of a quarter turn: there the small one of sine and cosine shows the
    angle's error, however coarse BF16 is.  Bound: 2^-25 of a turn, BF16's half step, and sine's own 2^-22."""
    m = M()
    rot, page = 64, 65536
    pairs = rot // 2
    f, _ = m.mnw_rope_frequencies(rot, 1e4, device="cuda")
    rng = np.random.default_rng(low + 1)
    some = rng.integers(low, high, 200000)
    turns = [Fraction(float(x)) * INV_2PI for x in f.cpu().tolist()]
    at = []  # for every pair a position next to a whole turn and one next to a quarter
    for quarter in (0.0, 0.25):
        for t in turns:
            frac = (some.astype(np.uint64) * np.uint64(int(t * 2 ** 64) % 2 ** 64)).astype(np.float64) / 2.0 ** 64
            off = np.abs((frac - quarter + 0.5) % 1.0 - 0.5)
            at.append(int(some[int(off.argmin())]))
    B, most = len(at), (high + page - 1) // page
    table = torch.zeros((B, most), dtype=torch.int32, device="cuda")
    k, v = (torch.empty((1, 1, page, rot), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((B, 1, rot), dtype=torch.bfloat16, device="cuda")
    first, second = ((lambda i: i), (lambda i: i + pairs)) if layout == "half" else ((lambda i: 2 * i), (lambda i: 2 * i + 1))
    for i in range(pairs):
        q[:, 0, first(i)] = 1.0
    kv = torch.zeros((B, 1, rot), dtype=torch.bfloat16, device="cuda")
    got = m.mnw_kv_append(q, kv, kv, k, v, table, _ints([p + 1 for p in at]), inv_freq=f,
                          layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED).double().cpu()[:, 0]
    for b, p in enumerate(at):
        i = b % pairs
        t = p * turns[i]
        a = float(2 * (t - round(t)) / (2 * INV_2PI))  # radians, in [-pi, pi]
        for x, want in ((first(i), np.cos(a) if b < pairs else float(np.sin(np.pi / 2 - a))), (second(i), np.sin(a))):
            tol = 2.0 ** -8 * abs(want) + 2 * np.pi * 2.0 ** -25 + 2.0 ** -22 * abs(want)
            assert abs(got[b, x].item() - want) <= tol, (p, i, got[b, x].item(), want)


def test_rotation_of_odd_frequencies():
    """Negative, zero, tiny, large and NaN entries of the table."""
    m = M()
    f = torch.tensor([-0.5, 0.0, -0.0, 1e-30, 1e-42, 100.0, float("nan"), 1.0], device="cuda")
    k, v = (torch.zeros((1, 1, 64, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, kv = _randn((5, 1, 64), 3), _randn((5, 1, 64), 4)
    got = m.mnw_kv_append(q, kv, kv, k, v, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), _ints([37]), inv_freq=f)
    ref, size = U.rotate_plain(q, np.arange(32, 37), f, 16, "half", 1.0)
    seen = torch.tensor([i for i in range(64) if i not in (6, 14)])
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size
    assert ((got.double().cpu() - ref).abs() <= tol)[..., seen].all()
    assert torch.isnan(got[..., [6, 14]]).all()


# ---- prompt chunks: many row tiles over many key tiles ----


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("counts,lens,blk,d", [
    ([700], [700], 1, 128),               # into an empty cache
    ([512], [5000], 32, 128),             # behind cached positions
    ([300, 1, 450, 2], [300, 4000, 2100, 2], 1, 64),  # a mixed batch
    ([257], [6001], 1 << 20, 64),         # every row sees everything
])
def test_attention_of_prompt_chunks(fmt, counts, lens, blk, d):
    """Several row tiles of 128 query rows (4 query heads on one kv head: 32 tokens a tile) over up to 47 key tiles."""
    m = M()
    cache = U.Cache(lens, 64, 1, d, fmt, seed=41)
    q = _randn((sum(counts), 4, d), 42)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, blk, d ** -0.5,
                                q_start=_ints(U.starts_of(counts)), want_lse=True, err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == 0
    U.check_attention(out, lse, q, counts, cache, blk, d ** -0.5, lost=2.0 ** -38 if fmt == "int8" else 0.0)


# ---- pages smaller and larger than a tile, keys and values in one allocation ----


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [4, 8, 128, 256, 1024, 24])
@pytest.mark.parametrize("joint", [False, True])
def test_attention_page_sizes(fmt, d, page, joint):
    """Blocks (48 and 128 query rows a kv head) and single tokens over pages of every way of copying."""
    m = M()
    for counts, lens in (([32, 12], [1100, 257]), ([1, 1], [777, 2049])):
        cache = U.Cache(lens, page, 3, d, fmt, seed=page, joint=joint)
        q = _randn((sum(counts), 12, d), 44)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 8, d ** -0.5, want_lse=True,
                                    q_start=_ints(U.starts_of(counts)), err=err, **cache.kw())
        assert m.mnw_moe_read_error(err) == 0
        U.check_attention(out, lse, q, counts, cache, 8, d ** -0.5, lost=2.0 ** -38 if fmt == "int8" else 0.0)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 40])
def test_offsets_past_32_bits(fmt, n):
    """Pages behind 2^32 bytes (BF16: elements) of keys: tiles copied whole and row by row, and an append there."""
    m = M()
    page, Hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * Hkv * d) + 40
    small = U.Cache([300], page, Hkv, d, fmt, seed=2, shuffle=False)
    k, v = (torch.empty((n_pages,) + small.k.shape[1:], dtype=small.k.dtype, device="cuda") for _ in range(2))
    far = torch.arange(n_pages - 8, n_pages, device="cuda")[:5]
    k[far], v[far] = small.k[:5], small.v[:5]
    kw = {}
    if fmt == "int8":
        kw = {x: torch.empty((n_pages, Hkv, page), device="cuda") for x in ("k_scale", "v_scale")}
        kw["k_scale"][far], kw["v_scale"][far] = small.ks[:5], small.vs[:5]
    table = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    table[0, :5] = far.to(torch.int32)
    q = _randn((n, Hkv, d), 5)
    out, lse = m.mnw_attn_paged(q, k, v, table, small.cache_lens, 1, 0.09, want_lse=True, **kw)
    U.check_attention(out, lse, q, [n], small, 1, 0.09, lost=2.0 ** -38 if fmt == "int8" else 0.0)
    kv = _randn((n, Hkv, d), 6)
    m.mnw_kv_append(None, kv, kv, k, v, table, small.cache_lens, **kw)
    m.mnw_kv_append(None, kv, kv, small.k, small.v, small.table, small.cache_lens, **small.kw())
    assert torch.equal(k[far].view(torch.int8), small.k[:5].view(torch.int8))
    assert torch.equal(v[far].view(torch.int8), small.v[:5].view(torch.int8))
    if fmt == "int8":
        own = small.table_host[0, :5].long().cuda()
        assert torch.equal(kw["k_scale"][far, :, :44], small.ks[own][:, :, :44])
