"""The block attention's wait runs out without a fault: it gives up after its
limit, reports MNW_DEVERR_TIMEOUT, and another role's wait leaves through the
abort flag; the context stays usable."""
import ctypes
import time

import pytest
import torch


@pytest.mark.gpu
def test_polled_wait_that_nothing_completes_times_out():
    import quantized_moe_expert_routed_gb300 as M
    for limit_us in (2000, 50000, 500000):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        left_early = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        M.mnw_moe_selftest_polled_wait_timeout(limit_us, err, left_early)
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
        assert int(err.item()) == M.DEVERR_TIMEOUT
        # 64 retries before the clock is first read and between looks: a few hundred us; the launch itself
        assert limit_us * 1e-6 <= elapsed < limit_us * 1e-6 + 0.1
        # the second warp left through the abort flag, not its own 2 s limit
        assert int(left_early.item()) == 1
    x = torch.ones((3, 256), dtype=torch.bfloat16, device="cuda")
    assert torch.allclose(M.mnw_rmsnorm(x, x[0])[0].float(), x.float(), rtol=2.0 ** -7)


def test_polled_wait_selftest_refuses_bad_arguments():
    import quantized_moe_expert_routed_gb300 as M
    call, word = M.load().mnw_moe_selftest_polled_wait_timeout, ctypes.c_void_p(256)
    assert call(1000, None, word, None) == call(1000, word, None, None) == 1
    assert call(0, word, word, None) == call(2_000_000, word, word, None) == 1
