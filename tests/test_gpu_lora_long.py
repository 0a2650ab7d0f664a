"""Adapters of prompts in the lengths that they have: every CTA of the second product has several blocks of columns, and
the first product's ring of steps goes round more than twice."""
import pytest
import torch

from test_gpu_decode_ops import M
from test_gpu_lora import check, inputs

pytestmark = pytest.mark.gpu


def shares(T, H, N, R, n):
    """(blocks of columns of a CTA in the second product at least, steps of one in the first): the host's formulas."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = -(-T // 128)
    splits = max(1, min(2 * sms // tiles, H // 256, 16))
    blocks = -(-N // (192 if R <= 64 else 128))
    about = tiles + min(n, T // 128) // 2
    best = min(range(1, min(blocks, 64) + 1), key=lambda s: (-(-about * s // sms)) * (-(-blocks // s) + 1))
    return blocks // best, -(-H // 64) // splits


@pytest.mark.parametrize("pattern", ["random", "runs"])
@pytest.mark.parametrize("R", [16, 32, 64, 128])
@pytest.mark.parametrize("T,H,N,n", [(9000, 4096, 5000, 4), (9001, 4096, 4808, 9), (20000, 2056, 3336, 4)])
def test_prompts(T, H, N, n, R, pattern):
    m = M()
    blocks, steps = shares(T, H, N, R, n)
    assert blocks >= 3 and steps >= 9, (blocks, steps)
    y, x, a, b, ids = inputs(T, H, N, R, n, T + R, pattern)
    scale = torch.linspace(-2.0, 2.0, n, device="cuda")
    wide_x, wide_y = torch.full((T, H + 40), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, N + 24), 9.0, dtype=torch.bfloat16, device="cuda")
    xs, ys = wide_x[:, 16:16 + H], wide_y[:, 8:8 + N]
    xs.copy_(x)
    ys.copy_(y)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = m.mnw_lora_add(y, x, a, b, ids, scale=scale, err=err)
    check(got, y, x, a, b, ids, scale)
    assert torch.equal(got[ids == -1], y[ids == -1])
    for _ in range(3):  # in place, rows apart, the same bits
        ys.copy_(y)
        m.mnw_lora_add(ys, xs, a, b, ids, scale=scale, out=ys, err=err)
        assert torch.equal(ys, got)
    assert (wide_y[:, :8] == 9.0).all() and (wide_y[:, 8 + N:] == 9.0).all() and int(err.item()) == 0
