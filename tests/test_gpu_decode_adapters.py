"""The example decoder with low-rank adapters beside its projections and a cache in 4 bits: adapters, append, paged
attention and the expert layer together."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import int4_util as I4
import paged_util as U
from test_gpu_decode_example import _prompts, example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_attention_half_over_its_own_cache(example):  # noqa: F811
    """Outputs and statistics from the queries and the rows that the calls before left; tokens of sequences without an
    adapter are what they are without any."""
    model = example.Decoder(layers=1, adapters=3, rank=24)
    lens, new, ids = [64, 160, 96], [32, 96, 5], [2, -1, 0]
    gen = torch.Generator().manual_seed(5)
    halves = [[n - m for n, m in zip(lens, new)], new]
    ys = [torch.randn((sum(c), model.H), generator=gen).bfloat16().cuda() for c in halves]
    outs = []
    for with_adapters in (True, False):
        cache = example.PagedCache(1, 3, 256, 64, model.Hkv, model.d, bits=4)
        for counts, y in zip(halves, ys):  # a prompt, then the tokens that are checked
            cache.grow(counts)
            starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
            adapter = torch.tensor(ids, dtype=torch.int32).repeat_interleave(torch.tensor(counts)).cuda()
            q, o = model.attention(0, y, cache, starts, adapter if with_adapters else None)
        model.check()
        rows = []
        for b, L in enumerate(lens):
            pos = np.arange(L)
            pg, sl = cache.table_host[b].numpy()[pos // 64], pos % 64
            rows.append(tuple(torch.from_numpy(I4.values(c[0].cpu().numpy()[pg, :, sl], s[0].cpu().numpy()[pg, :, sl]))
                              for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))))
        seen = SimpleNamespace(rows=rows, lens=lens, Hkv=model.Hkv, d=model.d, fmt="int4")
        _, lse, _, _, _ = U.attend_plain(q.cpu(), new, seen, model.block, model.d ** -0.5)
        U.check_attention(o, lse, q, new, seen, model.block, model.d ** -0.5, lost=2.0 ** -30)
        outs.append((q, o))
    base = slice(new[0], new[0] + new[1])
    for a, b in zip(*outs):
        assert torch.equal(a[base], b[base])
        assert not torch.equal(a[:new[0]], b[:new[0]])


def test_graph_writes_what_eager_calls_write(example):  # noqa: F811
    model = example.Decoder(adapters=4, rank=8)
    prompts = _prompts(model.vocab, (32, 128, 64))
    kw = dict(blocks=3, passes=2, bits=4, adapters=[3, -1, 0])
    eager = example.write(model, prompts, graph=False, **kw)
    graph = example.write(model, prompts, **kw)
    assert eager.shape == (3, 96) and torch.equal(eager, graph)
    other = example.write(model, prompts, **dict(kw, adapters=[1, -1, 0]))
    assert not torch.equal(other[0], graph[0])
