"""The decode step's operators refuse bad arguments on the host, before anything is launched (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 4
F = ctypes.c_float
P = ctypes.c_void_p
BIG = P(1 << 20)  # aligned, never dereferenced: the checks come first


@pytest.fixture(scope="module")
def lib():
    import quantized_moe_expert_routed_gb300 as M
    return M.load()


def norm(lib, **kw):
    a = dict(x=BIG, xs=256, r=None, w=BIG, T=2, H=256, eps=1e-6, ro=None, y=BIG, c=None, s=None)
    a.update(kw)
    return lib.mnw_rmsnorm(a["x"], a["xs"], a["r"], a["w"], a["T"], a["H"], F(a["eps"]), a["ro"], a["y"], a["c"], a["s"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, x=None, w=None), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=12, xs=16), INVALID),
    (dict(xs=128), INVALID), (dict(xs=260), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(x=P(8)), INVALID),
    (dict(y=None), INVALID), (dict(y=P(24)), INVALID), (dict(c=BIG), INVALID), (dict(s=BIG), INVALID),
    (dict(ro=BIG), INVALID), (dict(H=200, xs=200, c=BIG, s=BIG), UNSUPPORTED), (dict(H=16392, xs=16392), UNSUPPORTED),
])
def test_rmsnorm_refusals(lib, kw, want):
    assert norm(lib, **kw) == want


CACHE = dict(kc=BIG, vc=BIG, ks=None, vs=None, fmt=0, pages=8, page=16, stride=2 * 16 * 128, Hkv=2, d=128, table=BIG, most=4,
             lens=BIG, start=None, B=2, T=2, Hq=4, q=BIG, qs=512, err=None)


def append(lib, **kw):
    a = dict(CACHE, k=BIG, kst=256, v=BIG, vst=256, f=BIG, rot=128, layout=0, ms=1.0, qo=BIG)
    a.update(kw)
    return lib.mnw_kv_append(a["q"], a["qs"], a["k"], a["kst"], a["v"], a["vst"], a["B"], a["T"], a["Hq"], a["Hkv"], a["d"],
                             a["f"], a["rot"], a["layout"], F(a["ms"]), a["kc"], a["vc"], a["ks"], a["vs"], a["fmt"], a["pages"],
                             a["page"], a["stride"], a["table"], a["most"], a["lens"], a["start"], a["qo"], a["err"], None)


def attend(lib, **kw):
    a = dict(CACHE, blk=1, scale=0.1, out=BIG, lse=None, ws=BIG, wsb=1 << 40)
    a.update(kw)
    return lib.mnw_attn_paged(a["q"], a["qs"], a["B"], a["T"], a["Hq"], a["Hkv"], a["d"], a["kc"], a["vc"], a["ks"], a["vs"],
                              a["fmt"], a["pages"], a["page"], a["stride"], a["table"], a["most"], a["lens"], a["start"], a["blk"],
                              F(a["scale"]), a["out"], a["lse"], a["ws"], a["wsb"], a["err"], None)


BOTH = [
    (dict(T=0), OK), (dict(B=0), INVALID), (dict(B=-1), INVALID), (dict(T=-2), INVALID), (dict(T=3), INVALID),
    (dict(fmt=2), INVALID), (dict(fmt=1), INVALID), (dict(fmt=1, ks=BIG), INVALID), (dict(pages=0), INVALID),
    (dict(page=0), INVALID), (dict(page=1 << 17, stride=1 << 40), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(stride=2 * 16 * 128 - 8), INVALID), (dict(stride=2 * 16 * 128 + 4), INVALID),
    (dict(fmt=1, ks=BIG, vs=BIG, stride=2 * 16 * 128 + 8), INVALID), (dict(kc=None), INVALID), (dict(vc=P(8)), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(lens=P(2)), INVALID), (dict(start=P(6)), INVALID),
    (dict(most=0), INVALID), (dict(most=1 << 28), UNSUPPORTED), (dict(qs=504), INVALID), (dict(qs=516), INVALID),
    (dict(q=P(8)), INVALID), (dict(Hkv=0), INVALID),
]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(rot=144), INVALID), (dict(rot=-16), INVALID), (dict(rot=24), UNSUPPORTED), (dict(f=None), INVALID),
    (dict(layout=2), INVALID), (dict(ms=0.0), INVALID), (dict(ms=math.nan), INVALID), (dict(k=None), INVALID),
    (dict(v=P(8)), INVALID), (dict(kst=248), INVALID), (dict(vst=258), INVALID), (dict(qo=None), INVALID),
    (dict(Hq=0), INVALID),
])
def test_kv_append_refusals(lib, kw, want):
    assert append(lib, **kw) == want


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(Hq=3, qs=384), INVALID), (dict(blk=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.inf), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ws=P(128)), INVALID), (dict(wsb=1000), SMALL), (dict(lse=P(2)), INVALID),
    (dict(q=None), INVALID),
])
def test_attn_paged_refusals(lib, kw, want):
    assert attend(lib, **kw) == want


def test_workspace_size(lib):
    f = lib.mnw_attn_paged_workspace_size
    assert f(0, 1, 4, 2, 128) == f(1, 0, 4, 2, 128) == f(1, 1, 4, 3, 128) == 0
    assert 0 < f(1, 1, 4, 4, 128) <= f(1, 32, 16, 4, 128)
    assert f(4, 4, 16, 4, 128) % 256 == 0


def test_the_binding_refuses_before_the_library(lib):
    import quantized_moe_expert_routed_gb300 as M
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(M.MnwError):
        M.mnw_rmsnorm(x, x[0])  # not on a GPU
    with pytest.raises(M.MnwError):
        M.mnw_attn_paged(x, x, x, x, x, 1, 0.1)


def test_rope_frequencies(lib):
    import quantized_moe_expert_routed_gb300 as M
    f, m = M.mnw_rope_frequencies(128, 10000.0)
    want = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    assert m == 1.0 and np.array_equal(f.numpy(), want.astype(np.float32))
    lin, m = M.mnw_rope_frequencies(128, 10000.0, M.ROPE_SCALE_LINEAR, 8.0)
    assert m == 1.0 and np.array_equal(lin.numpy(), (want / 8.0).astype(np.float32))
    ntk, _ = M.mnw_rope_frequencies(128, 10000.0, M.ROPE_SCALE_NTK, 8.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1].item(), want[-1] / 8.0, rtol=1e-6)  # the slowest is divided by the factor
    parts, m = M.mnw_rope_frequencies(128, 10000.0, M.ROPE_SCALE_BY_PARTS, 8.0, 4096)
    assert np.isclose(m, 0.1 * math.log(8.0) + 1.0)
    ratio = parts.numpy() / want
    turns = want * 4096 / (2 * math.pi)
    assert np.allclose(ratio[turns > 33], 1.0, rtol=1e-6) and np.allclose(ratio[turns < 0.85], 1 / 8.0, rtol=1e-6)
    assert (np.diff(ratio) <= 1e-6).all()
    for bad in (dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=math.inf), dict(scale=4), dict(scale=1, factor=0.5),
                dict(scale=3, factor=2.0, original_len=0), dict(scale=3, factor=2.0, beta_fast=1.0), dict(scale=2, rot=2, factor=2.0)):
        with pytest.raises(M.MnwError):
            M.mnw_rope_frequencies(**{"rot": 64, **bad})
