"""The most tokens a rotary call can name."""
import torch
import pytest

import paged_kv_cache_121_gb300 as pa

pytestmark = pytest.mark.gpu


def test_two_to_the_31_less_one_tokens():
    """One head of one pair, in place, every angle zero and the factor two: doubled, the padding at the end left."""
    n = 2 ** 31 - 1
    x = torch.ones(n, 1, 2, dtype=torch.bfloat16, device="cuda")
    positions = torch.ones(n, dtype=torch.int32, device="cuda")
    positions[-2:] = -1
    pa.pa_rope(x, x, positions, torch.zeros(1, dtype=torch.float64, device="cuda"), factor=2.0)
    assert bool((x[:-2] == 2.0).all()) and bool((x[-2:] == 1.0).all())
    del x, positions
    torch.cuda.empty_cache()
