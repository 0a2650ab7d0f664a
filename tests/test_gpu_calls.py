"""The cache's and the adapters' calls in their native form and in Python: the same results, refusals and memory.  A given
stream goes through Python; without one the native form takes the call."""
import sys

import pytest
import torch

import int4_util as U4
import paged_util as U
from test_gpu_decode_ops import M, _randn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def both(f, *a, **kw):
    """Results of the native form and of the Python one."""
    return f(*a, **kw), f(*a, stream=torch.cuda.current_stream(), **kw)


def cache_of(fmt, lens, page, Hkv, d, seed, joint):
    c = U4.Cache(lens, page, Hkv, d, seed, joint=joint) if fmt == "int4" else U.Cache(lens, page, Hkv, d, fmt, seed, joint=joint)
    return c, {} if fmt == "bf16" else dict(k_scale=c.ks, v_scale=c.vs)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("n,Hq,Hkv,d,joint", [(1, 4, 1, 64, False), (3, 8, 2, 128, True)])
def test_attention(fmt, n, Hq, Hkv, d, joint):
    m = M()
    lens = [40, 7, 300]
    c, kw = cache_of(fmt, lens, 16, Hkv, d, 11, joint)
    wide = _randn((len(lens) * n, Hq + 2 * Hkv, d), 12)
    q = wide[:, :Hq]
    args = (q, c.k, c.v, c.table, c.cache_lens, 1, d ** -0.5)
    assert m._load_calls().attn_paged(*args, kw.get("k_scale"), kw.get("v_scale"), None, None, None, True, None, None) is not NotImplemented
    (o1, l1), (o2, l2) = both(m.mnw_attn_paged, *args, want_lse=True, **kw)
    assert torch.equal(o1, o2) and torch.equal(l1, l2) and o1.shape == q.shape and l1.shape == q.shape[:2]
    assert o1.dtype is BF16 and l1.dtype is torch.float32 and o1.is_contiguous()
    o = m.mnw_attn_paged(*args, **kw)
    assert torch.is_tensor(o) and torch.equal(o, o2)
    # everything given; integers for the scale; token ranges
    out, lse = torch.empty_like(o2), torch.empty_like(l2)
    ws = torch.empty(m.mnw_attn_paged_workspace_size(len(lens), q.shape[0], Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.arange(len(lens) + 1, dtype=torch.int32, device="cuda") * n
    got = m.mnw_attn_paged(*args, q_start=start, out=out, lse=lse, ws=ws, err=err, **kw)
    assert got[0] is out and got[1] is lse and torch.equal(out, o2) and torch.equal(lse, l2) and int(err) == 0
    one = both(m.mnw_attn_paged, *args[:6], 1, **kw)
    assert torch.equal(*one)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_append(fmt):
    m = M()
    Hq, Hkv, d, n = 4, 2, 64, 5
    c, kw = cache_of(fmt, [40, 9], 16, Hkv, d, 21, False)
    qkv = _randn((2 * n, Hq + 2 * Hkv, d), 22)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    freq, scale = m.mnw_rope_frequencies(32, device="cuda")
    args = (q, k, v, c.k, c.v, c.table, c.cache_lens, freq, m.ROPE_INTERLEAVED, scale)
    held = lambda: [t.clone() for t in (c.k, c.v, *kw.values())]  # noqa: E731
    before = held()
    q1 = m.mnw_kv_append(*args, **kw)
    first = held()
    for t, b in zip((c.k, c.v, *kw.values()), before):
        t.copy_(b)
    q2 = m.mnw_kv_append(*args, stream=torch.cuda.current_stream(), **kw)
    assert torch.equal(q1, q2) and q1.is_contiguous()
    for a, b, old in zip(first, held(), before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and not torch.equal(a.view(torch.uint8), old.view(torch.uint8))
    out = torch.empty_like(q1)
    assert m.mnw_kv_append(*args, q_out=out, **kw) is out and torch.equal(out, q1)
    assert m.mnw_kv_append(None, *args[1:], **kw) is None
    for a, b in zip(first, held()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("joint", [False, True])
def test_values(fmt, joint):
    m = M()
    c, kw = cache_of(fmt, [40, 9], 16, 2, 64, 31, joint)
    a, b = both(m.mnw_kv_values, c.v, kw["v_scale"])
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and a.shape == (c.v.shape[0], 2, 16, 64)
    out = torch.empty_like(a)
    assert m.mnw_kv_values(c.v, kw["v_scale"], out=out) is out and torch.equal(out.view(torch.int16), a.view(torch.int16))


@pytest.mark.parametrize("T", [1, 9, 1200])
def test_adapters(T):
    m = M()
    H, N, R = 64, 40, 16
    y, x = _randn((T, N + 8), 41)[:, :N], _randn((T, H), 42)
    a, b = torch.nn.Parameter(_randn((3, R, H), 43)), torch.nn.Parameter(_randn((3, N, R), 44))  # (as a module holds them)
    ids = (torch.arange(T, device="cuda") % 4 - 1).to(torch.int32)
    scale, ranks = torch.tensor([0.5, 1.0, 2.0], device="cuda"), torch.tensor([16, 8, 3], dtype=torch.int32, device="cuda")
    p, r = both(m.mnw_lora_add, y, x, a, b, ids, scale, ranks)
    assert torch.equal(p, r) and p.shape == (T, N) and not p.requires_grad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, m.mnw_lora_workspace_size(T, H, R, 3)), dtype=torch.uint8, device="cuda")
    assert m.mnw_lora_add(y, x, a, b, ids, scale, ranks, out=y, ws=ws, err=err) is y and torch.equal(y, r) and int(err) == 0


def test_results_and_scratch_are_given_back():
    m = M()
    c, kw = cache_of("int4", [500], 16, 1, 64, 51, False)
    q = _randn((1, 4, 64), 52)
    y, x, a, b = _randn((1100, 64), 53), _randn((1100, 64), 54), _randn((1, 8, 64), 55), _randn((1, 64, 8), 56)
    ids = torch.zeros(1100, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")

    def step():
        m.mnw_attn_paged(q, c.k, c.v, c.table, c.cache_lens, 1, 0.1, want_lse=True, **kw)
        m.mnw_attn_paged(q, c.k, c.v, c.table, c.cache_lens, 1, 0.1, out=out, lse=lse, **kw)
        m.mnw_lora_add(y, x, a, b, ids)
        m.mnw_kv_values(c.k, c.ks)
        m.mnw_kv_append(q, q[:, :1], q[:, 1:2], c.k, c.v, c.table, c.cache_lens, **kw)

    held = (q, c.k, c.ks, c.table, c.cache_lens, out, lse, y, x, a, b, ids)
    step()
    torch.cuda.synchronize()
    memory, counts = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in held]
    for _ in range(50):
        step()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == memory and [sys.getrefcount(t) for t in held] == counts


def test_refusals_are_the_same():
    m = M()
    c, kw = cache_of("int4", [40], 16, 1, 64, 61, False)
    q = _randn((1, 4, 64), 62)
    ok = dict(q=q, k_cache=c.k, v_cache=c.v, block_table=c.table, cache_lens=c.cache_lens, blk=1, scale=0.1, **kw)
    bad = [dict(blk=0), dict(q=q.float()), dict(q=q[:, :, :32]), dict(v_cache=c.v[1:]), dict(k_scale=None), dict(k_scale=c.ks[1:]),
           dict(block_table=c.table.long()), dict(cache_lens=c.cache_lens.repeat(2)), dict(out=torch.empty_like(q).float()),
           dict(lse=torch.empty(1, 5, device="cuda")), dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
           dict(q_start=c.cache_lens), dict(k_cache=c.k.transpose(2, 3), v_cache=c.v.transpose(2, 3)), dict(err=torch.zeros(1))]
    for b in bad:
        said = []
        for s in (None, torch.cuda.current_stream()):
            with pytest.raises(m.MnwError) as e:
                m.mnw_attn_paged(**{**ok, **b}, stream=s)
            said.append(str(e.value))
        assert said[0] == said[1], b
    y, x, a, bb = _randn((4, 64), 63), _randn((4, 64), 64), _randn((1, 8, 64), 65), _randn((1, 64, 8), 66)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for args in ((y, x[:3], a, bb, ids), (y, x, a[0], bb, ids), (y, x, a, bb[:, :32], ids), (y, x, a, bb, ids[:3]), (y, x, a[:, :4], bb[:, :, :4], ids),
                 (y, x, a, bb, ids.float()), (y.float(), x, a, bb, ids)):
        said = []
        for s in (None, torch.cuda.current_stream()):
            with pytest.raises(m.MnwError) as e:
                m.mnw_lora_add(*args, stream=s)
            said.append(str(e.value))
        assert said[0] == said[1]
    with pytest.raises(m.MnwError):
        m.mnw_lora_add(y, x, a, bb, ids, out=x)
    with pytest.raises(m.MnwError):
        m.mnw_kv_values(c.k, c.ks[1:])
    with pytest.raises(m.MnwError):
        m.mnw_kv_append(q, q[:, :2], q[:, :1], c.k, c.v, c.table, c.cache_lens, **kw)


def test_on_another_stream_and_in_inference_mode():
    m = M()
    c, kw = cache_of("int4", [400], 16, 1, 64, 71, False)
    q = _randn((1, 4, 64), 72)
    want = m.mnw_attn_paged(q, c.k, c.v, c.table, c.cache_lens, 1, 0.1, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.inference_mode():
        got = m.mnw_attn_paged(q, c.k, c.v, c.table, c.cache_lens, 1, 0.1, **kw)
        event = torch.cuda.Event()
        event.record()
    assert got.is_inference() and not want.is_inference()
    event.synchronize()
    assert torch.equal(got, want)
