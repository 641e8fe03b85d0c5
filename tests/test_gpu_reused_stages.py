"""Stages of the copy rings into which a kernel writes zeros by ordinary stores (V
rows past a context's end, rows of pages outside the pool) and which the next
copies overwrite: right, and the same bits on every run. Tolerances as derived in
prefill_cases."""
import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from prefill_cases import Case

pytestmark = pytest.mark.gpu

RUNS = 20


@pytest.mark.parametrize("dims", [(32, 8, 128, 16), (16, 16, 64, 0), (16, 4, 128, 64)])
def test_few_rows_prefill_tails(dims):
    """500 contexts of a few tiles, each ending inside one: every stage holds a mended tile again and again."""
    hq, hkv, d, bs = dims
    rng = np.random.default_rng(hq + d)
    ctx = (16 * rng.integers(0, 9, 500) + rng.integers(1, 16, 500)).tolist()
    c = Case([1 + i % 3 for i in range(500)], [n + 2 for n in ctx], hq, hkv, d, bs, "bf16", seed=3)
    ws = c.workspace()
    for causal in ((True, False) if bs else (False,)):
        out = c.run(causal, ws)
        c.check(out, causal)
        for _ in range(RUNS):
            assert torch.equal(c.run(causal, ws), out)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_balanced_decode_tails(d):
    rng = np.random.default_rng(d)
    ctx = (16 * rng.integers(0, 9, 500) + rng.integers(1, 16, 500)).tolist()
    c = Case([1] * 500, ctx, 32, 8, d, 16, "bf16", seed=4)
    assert pa.pa_decode_plan(500, 32, 8, d, 16, c.max_ctx, pa.PA_BF16, with_workspace=True)["balanced"] == 1
    n = pa.pa_decode_workspace_size(500, 32, 8, d, 16, c.max_ctx)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")

    def run():
        out = torch.full_like(c.query, 5.0)
        pa.pa_decode(out, c.query, c.kc, c.vc, c.tables_d, c.ctx_d, c.max_ctx, c.scale, workspace=ws)
        return out

    out = run()
    c.check(out, True)
    for _ in range(RUNS):
        assert torch.equal(run(), out)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("bs", [1, 2, 4])
def test_decode_pages_outside_the_pool(bs):
    """Blocks gathered row by row, every third page outside the pool: their tokens are zero keys and values."""
    c = Case([1] * 3, [700, 65, 1000], 8, 2, 128, bs, "bf16", seed=5)
    for b, n in enumerate(c.ctx_lens):
        for page in range(b, n // bs, 3):
            c.tables_d[b, page] = -1 if page % 2 else 10 ** 6
            c.k[b][page * bs:page * bs + bs] = 0
            c.v[b][page * bs:page * bs + bs] = 0

    def run():
        out = torch.full_like(c.query, 5.0)
        pa.pa_decode(out, c.query, c.kc, c.vc, c.tables_d, c.ctx_d, c.max_ctx, c.scale)
        return out

    out = run()
    c.check(out, True)
    for _ in range(RUNS):
        assert torch.equal(run(), out)
    assert pa.pa_device_status() == 0
