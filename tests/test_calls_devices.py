"""Tensors of a call on different devices, or on another than the current one, are refused by name and nothing is launched
(no GPU needed: stand-ins for tensors, which the native form leaves to the Python one)."""
import pytest

import call_stubs as C
import quantized_moe_expert_routed_gb300 as M


@pytest.mark.parametrize("name", C.CALLS)
def test_on_one_device(name, monkeypatch):
    tensors, rest = C.arguments(name)
    lib = C.install(monkeypatch)
    getattr(M, name)(**tensors, **rest)
    assert [c[0] for c in lib.calls] == [name]


@pytest.mark.parametrize("name", C.CALLS)
def test_a_tensor_elsewhere(name, monkeypatch):
    for which in C.arguments(name)[0]:
        with monkeypatch.context() as patch:
            tensors, rest = C.arguments(name)
            lib = C.install(patch)
            tensors[which].index = 1
            with pytest.raises(M.MnwError, match="device") as e:
                getattr(M, name)(**tensors, **rest)
            if which != C.FIRST[name]:
                assert str(e.value).startswith(which + ":"), which
            assert not lib.calls


@pytest.mark.parametrize("name", C.CALLS)
def test_all_on_another_device_than_the_current_one(name, monkeypatch):
    tensors, rest = C.arguments(name)
    lib = C.install(monkeypatch, device=1)
    with pytest.raises(M.MnwError, match="current device"):
        getattr(M, name)(**tensors, **rest)
    assert not lib.calls


@pytest.mark.parametrize("name", C.CALLS)
def test_a_stream_of_another_device(name, monkeypatch):
    class Stream:
        device_index, cuda_stream = 1, 0
    tensors, rest = C.arguments(name)
    lib = C.install(monkeypatch)
    with pytest.raises(M.MnwError, match="stream"):
        getattr(M, name)(**tensors, **rest, stream=Stream)
    assert not lib.calls


@pytest.mark.parametrize("name", C.CALLS)
def test_a_stream_that_does_not_say_its_device(name, monkeypatch):
    class Stream:  # (another library's)
        cuda_stream = 77
    tensors, rest = C.arguments(name)
    lib = C.install(monkeypatch)
    getattr(M, name)(**tensors, **rest, stream=Stream)
    assert lib.calls[0][1][-1] == 77
