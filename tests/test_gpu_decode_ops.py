"""The decode step's operators on the GPU against plain 64-bit forms: RMS norm
with the residual and INT8 groups, rotated append to a paged cache, attention
of new tokens over it.

Tolerances count roundings: half a step of BF16 is 2^-8 of the value
(finfo.eps / 2), of FP16 2^-11; FP32 sums and angles are bounded beside each
check."""
import math

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


# ---- norm ----


@pytest.mark.parametrize("T,H", [(1, 8), (1, 128), (3, 256), (5, 1000), (2, 2048), (33, 2176), (7, 4096), (300, 640),
                                 (2, 5120), (2, 8192), (3, 8200), (2, 16384)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm_matches_plain(T, H, with_residual):
    x, w = _randn((T, H), T + H), (1 + _randn((H,), H, 0.2).float()).bfloat16()
    r = _randn((T, H), H + 1, 3.0) if with_residual else None
    int8 = H % 128 == 0
    y, ro, codes, scales = M().mnw_rmsnorm(x, w, 1e-5, residual=r, int8=int8)
    z = x.float()
    if with_residual:
        want = (x.float() + r.float()).bfloat16()
        assert torch.equal(ro, want)
        z = want.float()
    else:
        assert ro is None
    z = z.double().cpu()
    ref = z / (z.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double().cpu()
    # BF16's rounding, and FP32's: a sum of H squares in partial sums of at most 16 and two products
    tol = (2.0 ** -8 + 2.0 ** -18) * ref.abs()
    assert ((y.double().cpu() - ref).abs() <= tol).all()
    if int8:
        c, s = M().mnw_moe_quantize_act(M().ACT_INT8_G128, y)
        assert torch.equal(codes, c) and torch.equal(scales, s)


def test_rmsnorm_strided_rows_in_place_and_special_rows():
    m = M()
    wide = _randn((6, 3 * 512), 4)
    x = wide[:, 512:1024]
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    a = m.mnw_rmsnorm(x, w, 1e-6)[0]
    b = m.mnw_rmsnorm(x.contiguous(), w, 1e-6)[0]
    assert torch.equal(a, b)
    # the residual in place, then the output over x
    xc, r = x.contiguous(), _randn((6, 512), 5)
    want_y, want_r, want_c, want_s = m.mnw_rmsnorm(xc, w, 1e-6, residual=r, int8=True)
    y, ro, c, s = m.mnw_rmsnorm(xc, w, 1e-6, residual=r, residual_out=r, y=xc, int8=True)
    assert ro is r and y is xc
    assert torch.equal(y, want_y) and torch.equal(r, want_r) and torch.equal(c, want_c) and torch.equal(s, want_s)
    # a zero row: zeros out, scale 0; a row with eps alone in the denominator; a NaN stays in its row
    z = torch.zeros((3, 512), dtype=torch.bfloat16, device="cuda")
    z[1] = 1e-20
    z[2, 7] = float("nan")
    y, _, c, s = m.mnw_rmsnorm(z, w, 1e-6, int8=True)
    assert (y[0] == 0).all() and (c[0] == 0).all() and (s[0] == 0).all()
    assert torch.allclose(y[1].float(), torch.full((512,), 1e-17, device="cuda"), rtol=2.0 ** -7)
    assert torch.isnan(y[2]).all()


def test_rmsnorm_codes_at_the_ends_of_the_range():
    """Groups from subnormal (whose scales hold few bits) to huge: the codes are those of y, bit for bit."""
    H = 1024
    x = _randn((40, H), 3)
    w = torch.tensor([2.0 ** e for e in (-133, -130, -126, -120, -100, 0, 60, 122)]).repeat_interleave(128)
    y, _, codes, scales = M().mnw_rmsnorm(x, w.bfloat16().cuda(), 1e-5, int8=True)
    assert torch.isfinite(y.float()).all()
    want, ws = U.quantise_rows(y.float().cpu().view(40, -1, 128).numpy())
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(codes.cpu().numpy().reshape(want.shape), want)


def test_rmsnorm_one_row_of_a_wider_tensor():
    """A single row's stride is not looked at, whatever the tensor it was cut from."""
    big = _randn((4, 1003), 4)
    x, w = big[:1, :1000], _randn((1000,), 5)
    assert torch.equal(M().mnw_rmsnorm(x, w)[0], M().mnw_rmsnorm(x.clone(), w)[0])


# ---- append ----


APPEND = [
    # counts, lens, page, Hq, Hkv, d, rot, layout, ragged
    ([1, 1, 1], [1, 17, 900], 16, 8, 2, 128, 128, "half", False),
    ([4, 4], [4, 70], 16, 4, 4, 128, 64, "interleaved", False),
    ([32, 32, 32], [32, 100, 5000], 64, 16, 4, 128, 32, "half", False),
    ([3, 0, 9, 1], [8, 5, 9, 131], 5, 6, 2, 64, 64, "interleaved", True),
    ([200, 1], [300, 1], 100, 5, 1, 64, 32, "half", True),
    ([2], [3], 1, 2, 2, 128, 0, "half", False),
    ([7], [2000], 1024, 1, 1, 64, 16, "interleaved", False),
]


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"n{c[0]}-p{c[2]}-d{c[5]}-r{c[6]}{c[7][0]}")
def test_kv_append_matches_plain(case, fmt):
    m = M()
    counts, lens, page, Hq, Hkv, d, rot, layout, ragged = case
    cache = U.Cache(lens, page, Hkv, d, fmt, seed=5, joint=fmt == "bf16")
    T = sum(counts)
    qkv = _randn((T, Hq + 2 * Hkv, d), 6, 2.0)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    f, ms = (None, 1.0) if rot == 0 else m.mnw_rope_frequencies(rot, 1e4, m.ROPE_SCALE_BY_PARTS, 4.0, 512, device="cuda")
    start = torch.tensor(U.starts_of(counts), dtype=torch.int32, device="cuda") if ragged else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = [t.clone() for t in (cache.k, cache.v)]
    got = m.mnw_kv_append(q, k, v, cache.k, cache.v, cache.table, cache.cache_lens, inv_freq=f,
                          layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED, mscale=ms, q_start=start,
                          err=err, **cache.kw())
    assert int(err.item()) == 0
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(counts, lens)])
    seq = np.repeat(np.arange(len(lens)), counts)
    if rot:
        want_q, size_q = U.rotate_plain(q, pos, f, rot, layout, ms)
        want_k, size_k = U.rotate_plain(k, pos, f, rot, layout, ms)
    else:
        want_q, want_k = q.double().cpu(), k.double().cpu()
        size_q, size_k = torch.zeros_like(want_q), torch.zeros_like(want_k)

    def near(a, ref, size):
        # BF16's half step; the angle (2^-23 turns), sin and cos (2 ulp) and three FP32 roundings: below 2^-18
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size
        assert ((a.double().cpu() - ref).abs() <= tol).all(), float(((a.double().cpu() - ref).abs() - tol).max())
    near(got, want_q, size_q)
    pg, sl = cache.table_host[seq, pos // page].long().cuda(), torch.as_tensor(pos % page).cuda()
    kept = torch.ones((cache.k.shape[0], page), dtype=torch.bool, device="cuda")
    kept[pg, sl] = False
    if fmt == "bf16":
        k_new, v_new = cache.k[pg, :, sl], cache.v[pg, :, sl]
        near(k_new, want_k, size_k)
        assert torch.equal(v_new, v)
    else:
        plain = U.Cache(lens, page, Hkv, d, "bf16", seed=5)
        m.mnw_kv_append(None, k, v, plain.k, plain.v, plain.table, plain.cache_lens, inv_freq=f,
                        layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED, mscale=ms, q_start=start)
        where = plain.table_host[seq, pos // page].long().cuda()
        for codes, scales, rows in ((cache.k, cache.ks, plain.k), (cache.v, cache.vs, plain.v)):
            c, s = U.quantise_rows(rows[where, :, sl].float().cpu().numpy())
            assert np.array_equal(codes[pg, :, sl].cpu().numpy(), c)
            assert np.array_equal(scales[pg, :, sl].cpu().numpy(), s)
    for now, then in zip((cache.k, cache.v), before):  # nothing else was touched
        a = now.transpose(1, 2)[kept].view(torch.int8 if fmt == "int8" else torch.int16)
        b = then.transpose(1, 2)[kept].view(torch.int8 if fmt == "int8" else torch.int16)
        assert torch.equal(a, b)


@pytest.mark.parametrize("at", [1000, 131071, 16777217, 1 << 30])
def test_rotation_keeps_far_positions(at):
    """Angles at far positions, by a cache whose table sends every page to page 0."""
    m = M()
    page = 65536
    most = at // page + 1
    table = torch.zeros((1, most), dtype=torch.int32, device="cuda")
    k = v = torch.empty((1, 1, page, 64), dtype=torch.bfloat16, device="cuda")
    q = _randn((3, 2, 64), 1)
    kv = _randn((3, 1, 64), 2)
    f, _ = m.mnw_rope_frequencies(64, 1e4, device="cuda")
    lens = torch.tensor([at], dtype=torch.int32, device="cuda")
    for layout in ("half", "interleaved"):
        got = m.mnw_kv_append(q, kv, kv, k, v.clone(), table, lens, inv_freq=f,
                              layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED)
        ref, size = U.rotate_plain(q, np.arange(at - 3, at), f, 64, layout, 1.0)
        # a second FP32 rounding of the 2^-24-turn tail beyond 2^24 positions
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -17 * size
        assert ((got.double().cpu() - ref).abs() <= tol).all()


def test_kv_append_in_place_queries_and_bad_inputs_are_left_out():
    m = M()
    cache = U.Cache([40, 6], 16, 2, 128, "bf16", seed=1, stale=0.0)
    q, k, v = _randn((4, 4, 128), 1), _randn((4, 2, 128), 2), _randn((4, 2, 128), 3)
    f, _ = m.mnw_rope_frequencies(128, 1e4, device="cuda")
    want = m.mnw_kv_append(q, k, v, cache.k, cache.v, cache.table, cache.cache_lens, inv_freq=f)
    same = q.clone()
    got = m.mnw_kv_append(same, k, v, cache.k, cache.v, cache.table, cache.cache_lens, inv_freq=f, q_out=same)
    assert got is same and torch.equal(got, want)
    for lens, table, code in (([40, 1], cache.table, m.DEVERR_BAD_LENGTH),  # fewer positions than new tokens
                              ([-3, 6], cache.table, m.DEVERR_BAD_LENGTH),
                              ([10 ** 6, 6], cache.table, m.DEVERR_BAD_LENGTH | m.DEVERR_BAD_PAGE),
                              ([40, 6], torch.full_like(cache.table, 1000), m.DEVERR_BAD_PAGE),
                              ([40, 6], torch.full_like(cache.table, -1), m.DEVERR_BAD_PAGE)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kc, vc = torch.zeros_like(cache.k), torch.zeros_like(cache.v)
        m.mnw_kv_append(q, k, v, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), inv_freq=f, err=err)
        assert m.mnw_moe_read_error(err) & code == code
        written = int((kc != 0).any(-1).any(1).sum())
        assert written <= (3 if code & m.DEVERR_BAD_LENGTH else 0)


# ---- attention ----


ATTEND = [
    # counts, lens, page, Hq, Hkv, d, blk, ragged
    ([1], [1], 16, 4, 4, 128, 1, False),
    ([1], [777], 16, 16, 4, 128, 1, False),
    ([1, 1, 1, 1, 1], [15, 16, 64, 65, 1000], 16, 8, 2, 128, 1, False),
    ([1, 1], [5000, 3], 64, 8, 1, 64, 1, False),
    ([1, 1, 1], [300, 1, 129], 1, 4, 2, 64, 1, False),
    ([1, 1], [500, 257], 100, 32, 2, 128, 1, False),
    ([2, 2, 2], [2, 130, 67], 20, 10, 2, 128, 1, False),
    ([4, 4], [70, 4], 5, 8, 4, 64, 32, False),
    ([8, 8], [8, 400], 64, 16, 4, 128, 1, False),
    ([32, 32], [32, 352], 64, 16, 4, 128, 32, False),
    ([32, 32, 32], [97, 45, 640], 32, 8, 8, 64, 32, False),
    ([32], [200], 16, 8, 1, 128, 1 << 30, False),
    ([5, 0, 1, 40], [6, 9, 700, 41], 16, 12, 4, 128, 7, True),
    ([130, 3], [200, 3], 64, 4, 2, 128, 32, True),
    ([100], [100], 16, 4, 1, 64, 1, False),
]


def _attend(cache, counts, Hq, blk, ragged, seed=3, **kw):
    m = M()
    T = sum(counts)
    q = _randn((T, Hq + 3, cache.d), seed)[:, 1:Hq + 1]
    scale = cache.d ** -0.5
    start = torch.tensor(U.starts_of(counts), dtype=torch.int32, device="cuda") if ragged else None
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, blk, scale, q_start=start,
                                want_lse=True, **cache.kw(), **kw)
    return q, out, lse, scale


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"n{c[0]}-L{c[1]}-p{c[2]}-d{c[5]}")
def test_attn_paged_matches_plain(case, fmt):
    counts, lens, page, Hq, Hkv, d, blk, ragged = case
    cache = U.Cache(lens, page, Hkv, d, fmt, seed=7, joint=page == 20)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, out, lse, scale = _attend(cache, counts, Hq, blk, ragged, err=err)
    assert int(err.item()) == 0
    U.check_attention(out, lse, q, counts, cache, blk, scale)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_attn_paged_long_split_and_many_sequences(fmt):
    # one long sequence over all CTAs; then more sequences than a CTA has threads
    cache = U.Cache([40003], 64, 2, 128, fmt, seed=8)
    q, out, lse, scale = _attend(cache, [1], 8, 1, False)
    U.check_attention(out, lse, q, [1], cache, 1, scale)
    lens = [1 + (37 * i) % 90 for i in range(700)]
    cache = U.Cache(lens, 16, 1, 64, fmt, seed=9)
    q, out, lse, scale = _attend(cache, [1] * 700, 2, 1, False)
    U.check_attention(out, lse, q, [1] * 700, cache, 1, scale)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_attn_paged_rows_that_see_nothing_and_bad_inputs(fmt):
    m = M()
    cache = U.Cache([0, 40, 2], 16, 2, 128, fmt, seed=4)
    q = _randn((9, 4, 128), 2)
    start = torch.tensor([0, 3, 6, 9], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.1, q_start=start, want_lse=True,
                                err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_LENGTH  # 0 and 2 positions for 3 new tokens
    U.check_attention(out, lse, q, [3, 3, 3], cache, 1, 0.1)
    assert (out[:3] == 0).all() and torch.isinf(lse[:3]).all() and (out[6] == 0).all()
    for lens, table, code in (([0, 10 ** 6, 2], cache.table, m.DEVERR_BAD_LENGTH),
                              ([0, -5, 2], cache.table, m.DEVERR_BAD_LENGTH),
                              ([0, 40, 3], torch.full_like(cache.table, 99999), m.DEVERR_BAD_PAGE),
                              ([0, 40, 3], torch.full_like(cache.table, -2), m.DEVERR_BAD_PAGE)):
        err.zero_()
        out = m.mnw_attn_paged(q, cache.k, cache.v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1, 0.1,
                               q_start=start, err=err, **cache.kw())
        assert m.mnw_moe_read_error(err) & code
        if code == m.DEVERR_BAD_PAGE:
            assert (out == 0).all()  # bad pages read as zeros
    # rows of no sequence are not written, a q_start out of range is brought back
    bad_start = torch.tensor([0, 3, 2, 50], dtype=torch.int32, device="cuda")
    err.zero_()
    m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.1, q_start=bad_start, err=err, **cache.kw())
    assert m.mnw_moe_read_error(err) & m.DEVERR_BAD_LENGTH


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_attn_paged_extreme_scores_and_scales(fmt):
    """Scores far from zero in both directions, keys growing along the cache, one dominant key; INT8 value scales over
    many powers of two and rows of zeros."""
    m = M()
    cache = U.Cache([600, 90], 16, 1, 128, fmt, seed=12)
    grow = torch.linspace(0.01, 30.0, 600).double()
    for b, L in enumerate(cache.lens):
        pos = torch.arange(L)
        pg, sl = cache.table_host[b, pos // 16].long().cuda(), (pos % 16).cuda()
        k, v = cache.rows[b]
        if fmt == "bf16":
            kk = (k * grow[:L, None, None]).bfloat16()
            kk[L // 2] = 0
            cache.k[pg, :, sl] = kk.cuda()
            cache.rows[b] = (kk.double(), v)
        else:
            f = grow[:L].float()
            f[L // 2] = 0
            ks = cache.ks[pg, :, sl].cpu() * f[:, None]
            vs = cache.vs[pg, :, sl].cpu() * torch.exp2((torch.arange(L) % 40 - 30).float())[:, None]
            vs[L // 3] = 0
            cache.ks[pg, :, sl], cache.vs[pg, :, sl] = ks.cuda(), vs.cuda()
            kc, vc = cache.k[pg, :, sl].cpu().double(), cache.v[pg, :, sl].cpu().double()
            cache.rows[b] = (kc * ks.double()[..., None], vc * vs.double()[..., None])
    for size in (1e-3, 1.0, 8.0):
        q = _randn((2, 4, 128), 3, size)
        q[0, 1] = 0
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.2, want_lse=True, **cache.kw())
        U.check_attention(out, lse, q, [1, 1], cache, 1, 0.2)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_attn_paged_blocks_long_split(fmt):
    """32-token blocks of one long and one short sequence: runs end inside items, several parts a row."""
    cache = U.Cache([9001, 77], 64, 2, 128, fmt, seed=18)
    q, out, lse, scale = _attend(cache, [32, 32], 8, 32, False)
    U.check_attention(out, lse, q, [32, 32], cache, 32, scale)
    # many small items in one run: segments of a single tile
    lens = [33 + (41 * i) % 200 for i in range(90)]
    cache = U.Cache(lens, 16, 4, 64, fmt, seed=19)
    q, out, lse, scale = _attend(cache, [9] * 90, 16, 4, False)
    U.check_attention(out, lse, q, [9] * 90, cache, 4, scale)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_attn_paged_blocks_extreme_scores_and_scales(fmt):
    """As for single tokens, with 40 query rows: keys growing along the cache, value scales over 40 powers of two, tiles
    of zero values after others.  The FP16 products of INT8 caches lose what is below 2^-38 of the row's largest."""
    m = M()
    cache = U.Cache([600, 290], 16, 1, 128, fmt, seed=22)
    grow = torch.linspace(0.01, 30.0, 600).double()
    for b, L in enumerate(cache.lens):
        pos = torch.arange(L)
        pg, sl = cache.table_host[b, pos // 16].long().cuda(), (pos % 16).cuda()
        k, v = cache.rows[b]
        if fmt == "bf16":
            kk = (k * grow[:L, None, None]).bfloat16()
            kk[L // 2] = 0
            cache.k[pg, :, sl] = kk.cuda()
            cache.rows[b] = (kk.double(), v)
        else:
            f = grow[:L].float()
            f[L // 2] = 0
            ks = cache.ks[pg, :, sl].cpu() * f[:, None]
            vs = cache.vs[pg, :, sl].cpu() * torch.exp2((torch.arange(L) % 40 - 30).float())[:, None]
            if b == 1:
                vs[128:256] = 0
            cache.ks[pg, :, sl], cache.vs[pg, :, sl] = ks.cuda(), vs.cuda()
            kc, vc = cache.k[pg, :, sl].cpu().double(), cache.v[pg, :, sl].cpu().double()
            cache.rows[b] = (kc * ks.double()[..., None], vc * vs.double()[..., None])
    for size in (1e-3, 1.0, 8.0):
        q = _randn((20, 4, 128), 3, size)
        q[0, 1] = 0
        out, lse = m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.2, want_lse=True, **cache.kw())
        U.check_attention(out, lse, q, [10, 10], cache, 1, 0.2, lost=2.0 ** -38 if fmt == "int8" else 0.0)


def test_attn_paged_offsets_past_32_bits():
    m = M()
    page, Hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * Hkv * d) + 40  # more than 2^32 elements
    k = torch.empty((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = U.Cache([300], page, Hkv, d, "bf16", seed=2, shuffle=False)
    far = torch.arange(n_pages - 8, n_pages, device="cuda")[:5]
    k[far], v[far] = small.k[:5], small.v[:5]
    table = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    table[0, :5] = far.to(torch.int32)
    q = _randn((1, 8, d), 5)
    out, lse = m.mnw_attn_paged(q, k, v, table, small.cache_lens, 1, 0.09, want_lse=True)
    U.check_attention(out, lse, q, [1], small, 1, 0.09)
    # and an append there
    kv = _randn((1, Hkv, d), 6)
    m.mnw_kv_append(None, kv, kv, k, v, table, small.cache_lens)
    assert torch.equal(k[far[299 // page], :, 299 % page], kv[0]) and torch.equal(v[far[299 // page], :, 299 % page], kv[0])


def test_decode_ops_streams_graph_and_repeat():
    """The same bits on another stream, with a dirty workspace, and from a captured graph replayed on new inputs."""
    m = M()
    cache = U.Cache([1000, 333], 16, 4, 128, "bf16", seed=3)
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    f, _ = m.mnw_rope_frequencies(128, 1e4, device="cuda")
    x, qkv = _randn((2, 512), 1), _randn((2, 16 + 8, 128), 2)
    ws = torch.full((m.mnw_attn_paged_workspace_size(2, 2, 16, 4, 128),), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 16, 128), dtype=torch.bfloat16, device="cuda")
    qo, y = torch.empty_like(out), torch.empty_like(x)

    def step(stream=None):
        m.mnw_rmsnorm(x, w, y=y, stream=stream)
        m.mnw_kv_append(qkv[:, :16], qkv[:, 16:20], qkv[:, 20:], cache.k, cache.v, cache.table, cache.cache_lens,
                        inv_freq=f, q_out=qo, stream=stream)
        m.mnw_attn_paged(qo, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.09, out=out, ws=ws, stream=stream)
        return [t.clone() for t in (y, qo, out)]
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # results allocated inside the call belong to the given stream
    r = m.mnw_attn_paged(qo, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.09, stream=side)
    side.synchronize()
    assert torch.equal(r, want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mnw_rmsnorm(x, w, y=y)
        m.mnw_kv_append(qkv[:, :16], qkv[:, 16:20], qkv[:, 20:], cache.k, cache.v, cache.table, cache.cache_lens,
                        inv_freq=f, q_out=qo)
        m.mnw_attn_paged(qo, cache.k, cache.v, cache.table, cache.cache_lens, 1, 0.09, out=out, ws=ws)
    x.copy_(_randn((2, 512), 11))
    qkv.copy_(_randn((2, 24, 128), 12))
    cache.cache_lens.copy_(torch.tensor([900, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, qo, out)]
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# ---- the forms that large batches and middling row counts take ----


@pytest.mark.parametrize("H", [136, 1152, 4096])
def test_rmsnorm_many_rows(H):
    """Enough rows that a thread takes two words of one."""
    T = 3000
    x, r = _randn((T, H), H), _randn((T, H), H + 1, 3.0)
    w = (1 + _randn((H,), H + 2, 0.2).float()).bfloat16()
    y, ro, codes, scales = M().mnw_rmsnorm(x, w, 1e-5, residual=r, int8=H % 128 == 0)
    want = (x.float() + r.float()).bfloat16()
    assert torch.equal(ro, want)
    z = want.double()
    ref = z / (z.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    # BF16's rounding, and FP32's: a sum of H squares in partial sums of at most 16 and two products
    assert ((y.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -18) * ref.abs()).all()
    if H % 128 == 0:
        c, s = U.quantise_rows(y.float().cpu().view(T, -1, 128).numpy())
        assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy().reshape(c.shape), c)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("half", 64, 48), ("interleaved", 128, 32)])
def test_kv_append_many_tokens_as_few(fmt, layout, d, rot):
    """One call over ragged sequences with several tokens a CTA, and a call per sequence with one: the same bits."""
    m = M()
    counts, Hq, Hkv, page = [701, 1, 0, 898, 3], 6, 2, 20
    lens = [900, 1, 33, 898, 77]
    cache = U.Cache(lens, page, Hkv, d, fmt, seed=9, stale=0.0)
    T = sum(counts)
    q, k, v = _randn((T, Hq, d), 1), _randn((T, Hkv, d), 2), _randn((T, Hkv, d), 3)
    f, _ = m.mnw_rope_frequencies(rot, 1e4, device="cuda")
    kw = dict(inv_freq=f, layout=m.ROPE_HALF if layout == "half" else m.ROPE_INTERLEAVED)
    start = U.starts_of(counts)
    few = [t.clone() for t in (cache.k, cache.v)] + [None if t is None else t.clone() for t in (cache.ks, cache.vs)]
    got = m.mnw_kv_append(q, k, v, cache.k, cache.v, cache.table, cache.cache_lens,
                          q_start=torch.tensor(start, dtype=torch.int32, device="cuda"), **kw, **cache.kw())
    for b, n in enumerate(counts):
        if n:
            at = slice(start[b], start[b + 1])
            one = m.mnw_kv_append(q[at], k[at], v[at], few[0], few[1], cache.table[b:b + 1], cache.cache_lens[b:b + 1],
                                  k_scale=few[2], v_scale=few[3], **kw)
            assert torch.equal(got[at], one)
    assert torch.equal(cache.k, few[0]) and torch.equal(cache.v, few[1])
    if fmt == "int8":
        assert torch.equal(cache.ks, few[2]) and torch.equal(cache.vs, few[3])


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("page,d", [(16, 128), (20, 128), (64, 64)])
@pytest.mark.parametrize("counts,lens", [([5], [700]), ([8], [8]), ([7, 3, 11], [300, 3, 1111])])
def test_attn_paged_17_to_32_rows(fmt, page, d, counts, lens):
    cache = U.Cache(lens, page, 2, d, fmt, seed=len(lens))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, out, lse, scale = _attend(cache, counts, 8, 1, len(set(counts)) > 1, err=err)
    assert int(err.item()) == 0
    U.check_attention(out, lse, q, counts, cache, 1, scale)
