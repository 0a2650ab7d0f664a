"""The native form of the cache's and the adapters' calls leaves what it does not take to the Python one (no GPU needed)."""
import pytest
import torch

import quantized_moe_expert_routed_gb300 as M


@pytest.fixture(scope="module")
def native():
    return M._load_calls()


def test_what_is_not_a_plain_cuda_tensor_is_left_alone(native):
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    for o in (x, None, 3, "x", [x]):
        assert native.kv_values(o, o, None) is NotImplemented
        assert native.lora_add(o, o, o, o, o, None, None, None, None, None) is NotImplemented
        assert native.attn_paged(o, o, o, o, o, 1, 1.0, o, o, None, None, None, False, None, None) is NotImplemented
        assert native.kv_append(o, o, o, o, o, o, o, None, 0, 1.0, o, o, None, None, None) is NotImplemented


def test_numbers_of_arguments(native):
    for f in (native.kv_values, native.lora_add, native.attn_paged, native.kv_append):
        assert f() is NotImplemented and f(*[None] * 20) is NotImplemented
    with pytest.raises(TypeError):
        native.bind(1, 2)


def test_the_python_form_says_what_is_wrong():
    x, c = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 16, 32, dtype=torch.uint8)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(M.MnwError, match="k_cache and v_cache"):
        M.mnw_attn_paged(x, c, c, i, i[0], 1, 1.0, k_scale=c, v_scale=c)
    with pytest.raises(M.MnwError, match="k_cache and v_cache"):
        M.mnw_kv_append(x, x, x, c, c, i, i[0], k_scale=c, v_scale=c)
    with pytest.raises(M.MnwError, match="cache: expected a CUDA tensor"):
        M.mnw_kv_values(c, c)
    with pytest.raises(M.MnwError, match="y: expected a CUDA tensor"):
        M.mnw_lora_add(x[0], x[0], x, x, i[0])
