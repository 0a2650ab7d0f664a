"""A workspace whose elements do not lie side by side is refused: a call writes as many bytes from its address on as it has
elements (no GPU needed)."""
import pytest

import call_stubs as C
import quantized_moe_expert_routed_gb300 as M


@pytest.mark.parametrize("name", ["mnw_attn_paged", "mnw_lora_add"])
@pytest.mark.parametrize("shape,stride", [(lambda n: (n,), (2,)), (lambda n: (n,), (0,)), (lambda n: (2, n), (0, 1)),
                                          (lambda n: (n, 2), (1, 1 << 20))])
def test_strided_workspaces(name, shape, stride, monkeypatch):
    tensors, rest = C.arguments(name)
    n = tensors["ws"].numel()
    tensors["ws"] = C.Tensor(shape(n), C.U8, stride=stride)
    lib = C.install(monkeypatch)
    with pytest.raises(M.MnwError, match="^ws: expected a contiguous"):
        getattr(M, name)(**tensors, **rest)
    assert not lib.calls


@pytest.mark.parametrize("name", ["mnw_attn_paged", "mnw_lora_add"])
@pytest.mark.parametrize("shape", [lambda n: (n,), lambda n: (1, n), lambda n: (n + 1, 1), lambda n: (2, (n + 1) // 2)])
def test_contiguous_ones_of_any_shape(name, shape, monkeypatch):
    tensors, rest = C.arguments(name)
    tensors["ws"] = C.Tensor(shape(tensors["ws"].numel()), C.U8)
    lib = C.install(monkeypatch)
    getattr(M, name)(**tensors, **rest)
    assert [c[0] for c in lib.calls] == [name]
