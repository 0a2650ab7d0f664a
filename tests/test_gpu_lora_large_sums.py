"""Adapters whose finite inner sums lie above BF16's largest value (and below FP32's)."""
import pytest
import torch

from test_gpu_decode_ops import M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,R", [(1, 8), (40, 32), (300, 64), (300, 128), (2000, 16), (2000, 64), (1100, 128)])
def test_inner_sums_between_bf16s_largest_and_fp32s(T, R):
    """A x = +-(2^128 - 2^118), of two products, in half of the ranks: exactly B's 2^-20 of it, and nothing from the others."""
    H, N, n = 64, 72, 2
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 255 * 2.0 ** 57, 3 * 2.0 ** 55
    a = torch.zeros((n, R, H), dtype=torch.bfloat16, device="cuda")
    a[0, ::2, :2] = 2.0 ** 63  # 2^128 (1 - 2^-8) and 2^128 3 2^-10
    a[0, 1::2, 2] = 1.0
    a[1] = -a[0]
    b = torch.zeros((n, N, R), dtype=torch.bfloat16, device="cuda")
    b[:, :, 0] = 2.0 ** -20
    y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    ids = (torch.arange(T, device="cuda") % 2).to(torch.int32)
    got = M().mnw_lora_add(y, x, a, b, ids).double()
    want = (2.0 ** 128 - 2.0 ** 118) * 2.0 ** -20 * torch.where(ids == 0, 1.0, -1.0).double()[:, None]
    assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -16) * want.abs()).all()
