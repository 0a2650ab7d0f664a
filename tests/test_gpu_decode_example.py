"""The example decoder: norm, append, paged attention and the expert layer together."""
import os
import sys
from types import SimpleNamespace

import pytest
import torch

import paged_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    here = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    sys.path.insert(0, here)
    try:
        import decode_blocks
    finally:
        sys.path.remove(here)
    return decode_blocks


def _prompts(vocab, lens):
    g = torch.Generator().manual_seed(3)
    return [torch.randint(vocab, (n,), generator=g).tolist() for n in lens]


def test_attention_half_over_its_own_cache(example):
    """Outputs and statistics from the queries and the cache rows that the calls before left."""
    model = example.Decoder(layers=1)
    lens, new = [64, 160], [32, 96]
    cache = example.PagedCache(1, 2, 256, 64, model.Hkv, model.d)
    gen = torch.Generator().manual_seed(5)
    for counts in ([n - m for n, m in zip(lens, new)], new):  # a prompt, then the tokens that are checked
        cache.grow(counts)
        y = torch.randn((sum(counts), model.H), generator=gen).bfloat16().cuda()
        starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
        q, o = model.attention(0, y, cache, starts)
    model.check()
    rows = []
    for b, L in enumerate(lens):
        pos = torch.arange(L)
        pg, sl = cache.table_host[b, pos // 64].long(), pos % 64
        rows.append(tuple(c[0].cpu()[pg, :, sl].double() * s[0].cpu()[pg, :, sl].double()[..., None]
                          for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))))
    seen = SimpleNamespace(rows=rows, lens=lens, Hkv=model.Hkv, d=model.d, fmt="int8")
    _, lse, _, _, _ = U.attend_plain(q.cpu(), new, seen, model.block, model.d ** -0.5)
    U.check_attention(o, lse, q, new, seen, model.block, model.d ** -0.5, lost=2.0 ** -38)


def test_graph_writes_what_eager_calls_write(example):
    model = example.Decoder()
    prompts = _prompts(model.vocab, (32, 128, 64))
    eager = example.write(model, prompts, blocks=3, passes=2, graph=False)
    graph = example.write(model, prompts, blocks=3, passes=2)
    assert eager.shape == (3, 96) and torch.equal(eager, graph)
    assert int(eager.min()) >= 0 and int(eager.max()) < model.vocab and eager.unique().numel() > 8
