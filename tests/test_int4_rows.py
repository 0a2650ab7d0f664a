"""Cached rows in 4 bits on the host: the layout, and refusals of the calls that take them (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import int4_util as I4
from test_decode_refusals import BIG, INVALID, OK, UNSUPPORTED, P, append, attend, lib  # noqa: F401


def test_layout_and_rule():
    rng = np.random.default_rng(1)
    codes = rng.integers(-8, 8, (5, 64))
    assert np.array_equal(I4.unpack(I4.pack(codes)), codes)
    assert I4.pack(np.array([-8, -7, -8, -8, -8, -8, -8, -8])[None]).tolist() == [[0, 0, 1, 0]]  # element 1: bit 16
    x = (torch.randn((6, 128), dtype=torch.float64) * torch.logspace(-3, 1, 128)).bfloat16().double().numpy()
    data, rec = I4.quantise(x)
    # an element is off by half a code of its quarter at most
    step = (rec[:, 4:].astype(np.float64) * rec[:, :4].copy().view("<f4").astype(np.float64)).repeat(32, 1)
    assert (np.abs(I4.values(data, rec) - x) <= step / 2).all()
    assert np.abs(I4.unpack(data)).max() == 7


INT4 = dict(fmt=2, ks=BIG, vs=BIG)
BOTH = [(dict(INT4, T=0), OK), (dict(INT4, ks=None), INVALID), (dict(INT4, vs=None), INVALID), (dict(INT4, ks=P(4)), INVALID),
        (dict(INT4, stride=2 * 16 * 128 + 16), INVALID), (dict(INT4, stride=2 * 16 * 128 - 32), INVALID),
        (dict(INT4, kc=P(8)), INVALID), (dict(INT4, d=32), UNSUPPORTED), (dict(fmt=3, ks=BIG, vs=BIG), INVALID)]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("kw,want", BOTH)
def test_calls_on_a_cache_refuse(lib, call, kw, want):  # noqa: F811
    assert call(lib, **kw) == want


def values(lib, **kw):  # noqa: F811
    a = dict(c=BIG, s=BIG, fmt=2, pages=4, page=16, Hkv=2, d=128, stride=2 * 16 * 128, out=BIG)
    a.update(kw)
    return lib.mnw_kv_values(a["c"], a["s"], a["fmt"], a["pages"], a["page"], a["Hkv"], a["d"], ctypes.c_longlong(a["stride"]), a["out"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=0), INVALID), (dict(fmt=3), INVALID), (dict(c=None), INVALID), (dict(s=None), INVALID), (dict(s=P(4)), INVALID),
    (dict(c=P(8)), INVALID), (dict(out=None), INVALID), (dict(out=P(8)), INVALID), (dict(pages=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(stride=4000), INVALID), (dict(fmt=1, s=P(2)), INVALID), (dict(page=65537, stride=1 << 40), UNSUPPORTED),
])
def test_values_refuse(lib, kw, want):  # noqa: F811
    assert values(lib, **kw) == want


def test_the_binding_refuses(lib):  # noqa: F811
    import quantized_moe_expert_routed_gb300 as M
    x = torch.zeros((2, 1, 4, 64), dtype=torch.uint8)
    with pytest.raises(M.MnwError):
        M.mnw_kv_values(x, x)  # not on a GPU
    with pytest.raises(M.MnwError):
        M.mnw_kv_values(x.bfloat16(), None)
