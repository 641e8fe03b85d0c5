"""pa_prefill at the edges of its supported sizes and values; tolerances as derived
in prefill_cases."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from prefill_cases import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv", [16380, 16384, 65535])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_very_many_kv_heads(hkv, dt):
    """On both sides of what the few-rows kernel's merge can launch, and the most heads there may be."""
    c = Case([2, 1], [21, 5], hkv, hkv, 64, 16, dt, seed=1, spare=1)
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), True)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
