"""A warp that waits for a stage gives up as one: lanes that went on alone would
stand at the warp's next full-mask step for ever. pa_check_wait_timeout lets half
of a warp's lanes run out of time and completes the phase for the other half; a
warp that parts is reported as PA_ERR_CUDA in place of PA_ERR_TIMEOUT."""
import time

import pytest
import torch

import paged_kv_cache_121_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("timeout_us", [1000, 100_000])
def test_a_warp_gives_up_as_one(timeout_us):
    torch.cuda.synchronize()
    assert pa.pa_device_status(clear=True) == 0
    t0 = time.perf_counter()
    pa.pa_check_wait_timeout(timeout_us)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 2.0
    assert pa.pa_device_status(clear=True) == pa.PA_ERR_TIMEOUT
    assert pa.pa_device_status() == 0
