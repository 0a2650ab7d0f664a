"""Attention over the 4-bit cache where each CTA has many key tiles, and items that begin and end inside its run: the
rings go round several times, tiles copied whole and row by row follow each other, and sums are carried on."""
import pytest
import torch

import int4_device as D4
from test_gpu_decode_ops import M, _randn

pytestmark = pytest.mark.gpu


def run(cache, counts, Hq, blk, seed=1, q_scale=1.0, some=None, per=4, again=3, lost=D4.LOST):
    m = M()
    units, runs = D4.units_and_runs(counts, cache.lens, Hq // cache.Hkv, cache.Hkv)
    assert units >= per * runs, (units, runs)  # what the case is about
    q = _randn((sum(counts), Hq, cache.d), seed, q_scale)
    start = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: m.mnw_attn_paged(q, cache.k, cache.v, cache.table, cache.cache_lens, blk, cache.d ** -0.5,  # noqa: E731
                                    q_start=start, want_lse=True, err=err, **cache.kw())
    out, lse = call()
    for _ in range(again):  # the same bits, whatever the order of the CTAs
        o, l = call()
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)
    D4.check(out, lse, q, counts, cache, blk, cache.d ** -0.5, some=some, lost=lost)
    return m.mnw_moe_read_error(err)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,L", [(8, 150000), (64, 150001), (72, 90000), (128, 90000), (136, 90100), (256, 90000)])
def test_one_long_sequence(d, Hq, L):
    """1 and 8, 9 and 16, 17 and 32 query rows a kv head; runs end inside items."""
    cache = D4.Cache([L], 64, 8, d, seed=Hq)
    assert run(cache, [1], Hq, 1) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("G", [2, 12, 28])
def test_short_sequences_several_a_run(d, page, G):
    """Items of one and two tiles, partly filled: runs cross items, and whole tiles follow others of rows."""
    lens = [1 + 37 * i % 500 for i in range(320)]
    cache = D4.Cache(lens, page, 8, d, seed=G)
    assert run(cache, [1] * len(lens), 8 * G, 1, some=set(range(0, 320, 13)) | {319}) == 0


@pytest.mark.parametrize("d,L", [(64, 9000), (128, 4500)])
@pytest.mark.parametrize("page", [16, 20, 256])
def test_blocks(d, L, page):
    """16 refinement blocks of 32 tokens, 128 query rows a kv head; lengths that end inside tiles, some far shorter."""
    lens = [L - 61 * i for i in range(12)] + [32, 95, 1000, 129]
    cache = D4.Cache(lens, page, 4, d, seed=page)
    assert run(cache, [32] * 16, 16, 32, some={0, 3, 11, 12, 13, 14, 15}) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hq,L", [(1, 4, 120000), (1, 48, 60000), (1, 96, 60000), (32, 16, 30000)])
def test_values_and_scores_that_rise_along_the_cache(d, n, Hq, L):
    """The row's reference moves all the way, 24 powers of two by the values, and by scores that spread widely."""
    cache = D4.Cache([L, L // 2], 16, 4, d, seed=n + Hq, rising=24.0)
    assert run(cache, [n, n], Hq, 32, q_scale=4.0, per=2) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n,Hq", [(1, 8), (1, 40), (1, 96), (32, 16)])
def test_bad_pages_in_the_middle_of_runs(d, page, n, Hq):
    """Tiles row by row between tiles copied whole, anywhere in a run; two sequences have none and are untouched."""
    m = M()
    L = 40000 if n == 1 else 9000
    entries = [(0, e, v) for e, v in ((0, -1), (3, 10 ** 6), (40, -5), (41, 1 << 30), (100, -1))] + [(2, e, -1) for e in (17, 77)]
    cache = D4.Cache([L, L - 100, L - 3, 700], page, 4, d, seed=page, bad=entries)
    assert run(cache, [n] * 4, Hq, 32, per=1) == m.DEVERR_BAD_PAGE


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("counts,lens,blk", [([700], [700], 1), ([512], [20000], 32), ([300, 1, 450, 2], [300, 16000, 12100, 2], 1),
                                             ([257], [30001], 1 << 20)])
def test_prompt_chunks(d, counts, lens, blk):
    """Many row tiles over many key tiles, causal, by blocks, and unmasked."""
    cache = D4.Cache(lens, 64, 2, d, seed=41)
    assert run(cache, counts, 8, blk, per=0.5) == 0
