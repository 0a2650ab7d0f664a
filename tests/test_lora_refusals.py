"""The adapters' call refuses bad arguments on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from test_decode_refusals import BIG, INVALID, OK, SMALL, UNSUPPORTED, F, P, lib  # noqa: F401

LL = ctypes.c_longlong


def call(lib, **kw):  # noqa: F811
    v = dict(x=BIG, xs=256, a=BIG, b=BIG, s=None, r=None, n=4, R=16, i=BIG, T=3, H=256, N=128, y=BIG, ys=128, o=P(1 << 22), os=128,
             ws=BIG, wsb=1 << 40, err=None)
    v.update(kw)
    return lib.mnw_lora_add(v["x"], LL(v["xs"]), v["a"], v["b"], v["s"], v["r"], v["n"], v["R"], v["i"], v["T"], v["H"], v["N"], v["y"],
                            LL(v["ys"]), v["o"], LL(v["os"]), v["ws"], v["wsb"], v["err"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, x=None, ws=None), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(N=0), INVALID), (dict(R=0), INVALID),
    (dict(n=0), INVALID), (dict(n=1025), UNSUPPORTED), (dict(R=12), UNSUPPORTED), (dict(R=136), UNSUPPORTED), (dict(H=252), UNSUPPORTED),
    (dict(N=124), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 8, ys=1 << 21, os=1 << 21), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(i=None), INVALID), (dict(y=None), INVALID),
    (dict(o=None), INVALID), (dict(x=P(8)), INVALID), (dict(a=P(8)), INVALID), (dict(b=P(24)), INVALID),
    (dict(i=P(2)), INVALID), (dict(s=P(2)), INVALID), (dict(r=P(2)), INVALID), (dict(y=P(8)), INVALID), (dict(o=P(8)), INVALID),
    (dict(T=1100, ws=None), INVALID), (dict(T=1100, wsb=100), SMALL), (dict(ws=P(128)), INVALID), (dict(xs=248), INVALID), (dict(xs=260), INVALID), (dict(ys=120), INVALID), (dict(ys=132), INVALID),
    (dict(os=120), INVALID), (dict(os=132), INVALID), (dict(o=BIG, os=256), INVALID), (dict(x=P(1 << 23), o=P(1 << 23)), INVALID),
])
def test_refusals(lib, kw, want):  # noqa: F811
    assert call(lib, **kw) == want


def test_workspace_size(lib):  # noqa: F811
    f = lib.mnw_lora_workspace_size
    assert f(0, 256, 16, 4) == f(1, 0, 16, 4) == f(1, 256, 0, 4) == f(1, 256, 136, 4) == f(1, 256, 16, 0) == 0
    assert f(1, 256, 16, 4) == 0  # few tokens need none
    assert 0 < f(1100, 256, 16, 4) <= f(1100, 4096, 64, 4) and f(2000, 4096, 64, 4) % 256 == 0


def test_the_binding_refuses_before_the_library(lib):  # noqa: F811
    import quantized_moe_expert_routed_gb300 as M
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(M.MnwError):
        M.mnw_lora_add(x, x, x, x, x)  # not on a GPU
