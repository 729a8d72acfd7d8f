"""Two warps that barriers join, one of them late, on a wait that runs out (part of fp8_wait_selftest): both leave at
the same tile, within the limit, and the kernel ends.  The wait is bounded by itself; nothing faults or hangs."""
import time

import pytest
import torch

import fp8_delayed_scaling_03_b200 as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_ms", [1, 20])
def test_two_warps_give_up_together(limit_ms):
    assert F.fp8_get_device_status() == 0
    flag = torch.ones(1, dtype=torch.int32, device="cuda")
    for _ in range(5):
        res = torch.full((2,), 7, dtype=torch.int32, device="cuda")
        t0 = time.perf_counter()
        F.fp8_wait_selftest(flag, limit_ms * 1_000_000, res)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 10.0
        assert res.tolist() == [1, 0]    # -1: the two warps left at different tiles
        assert F.fp8_get_device_status() == F.FP8_ERR_DEVICE_TIMEOUT
    assert F.fp8_get_device_status() == 0
