"""The error word is four bytes at a multiple of four: a tensor without them is refused (no GPU needed)."""
import pytest
import torch

import call_stubs as C
import quantized_moe_expert_routed_gb300 as M

TAKE = ["mnw_kv_append", "mnw_attn_paged", "mnw_lora_add"]


@pytest.mark.parametrize("name", TAKE)
@pytest.mark.parametrize("shape,dtype,address", [((1,), C.U8, 1 << 20), ((1,), torch.float16, 1 << 20), ((3,), torch.int8, 1 << 20),
                                                 ((8,), C.U8, (1 << 20) + 1), ((2,), torch.int16, (1 << 20) + 2)])
def test_no_word(name, shape, dtype, address, monkeypatch):
    tensors, rest = C.arguments(name)
    tensors["err"] = C.Tensor(shape, dtype, address=address)
    lib = C.install(monkeypatch)
    with pytest.raises(M.MnwError, match="^err: expected a CUDA tensor"):
        getattr(M, name)(**tensors, **rest)
    assert not lib.calls


@pytest.mark.parametrize("name", TAKE)
@pytest.mark.parametrize("shape,dtype,address", [((), C.I32, 1 << 20), ((7,), C.I32, (1 << 20) + 4), ((4,), C.U8, 1 << 20),
                                                 ((1,), torch.int64, 1 << 20), ((0,), C.I32, 0)])
def test_words(name, shape, dtype, address, monkeypatch):
    tensors, rest = C.arguments(name)
    tensors["err"] = C.Tensor(shape, dtype, address=address)
    lib = C.install(monkeypatch)
    getattr(M, name)(**tensors, **rest)
    assert [c[0] for c in lib.calls] == [name]


@pytest.mark.parametrize("name", TAKE)
def test_on_the_host(name, monkeypatch):
    tensors, rest = C.arguments(name)
    tensors["err"] = torch.zeros(1, dtype=torch.int32)
    lib = C.install(monkeypatch)
    with pytest.raises(M.MnwError, match="^err: expected a CUDA tensor"):
        getattr(M, name)(**tensors, **rest)
    assert not lib.calls


def test_the_library_refuses_what_is_not_aligned():
    from test_decode_refusals import INVALID, P, append, attend
    from test_lora_refusals import call
    lib = M.load()
    for f in (append, attend, call):
        for at in (1, 2, (1 << 20) + 3):
            assert f(lib, err=P(at)) == INVALID
