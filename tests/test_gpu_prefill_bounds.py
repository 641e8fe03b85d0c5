"""Contexts longer than max_context_len, or than the block table reaches, under a
causal mask: what lies past the bound is not attended, and the mask still counts
from the context's own length. Tolerances as derived in prefill_cases."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from prefill_cases import Case

pytestmark = pytest.mark.gpu


def check(c, out, bound):
    """Token i of n sees the first min(context - n + i + 1, bound) tokens."""
    g = c.hq // c.hkv
    u = 0.0 if c.dt == torch.float32 else torch.finfo(c.dt).eps / 2
    for b in range(c.n):
        n, ctx, at = c.q_lens[b], c.ctx_lens[b], int(c.start[b])
        for i in range(n):
            sees = max(0, min(ctx - n + i + 1, bound))
            got = out[at + i].double()
            if sees == 0:
                assert not bool(got.any()), (b, i)
                continue
            q = c.query[at + i].double().view(c.hkv, g, c.d)
            k, v = c.k[b][:sees].double(), c.v[b][:sees].double()
            p = torch.softmax(torch.einsum("hgd,chd->hgc", q, k) * c.scale, -1)
            want = torch.einsum("hgc,chd->hgd", p, v).reshape(c.hq, c.d)
            avg = torch.einsum("hgc,chd->hgd", p, v.abs()).reshape(c.hq, c.d)
            size = torch.einsum("hgd,chd->hgc", q.abs(), k.abs()).amax(-1).reshape(c.hq, 1)
            tol = (u + 2 * (ctx + 16) * 2.0 ** -23 + 2 * (c.d + 2) * 2.0 ** -23 * abs(c.scale) * size) * avg
            if c.dt == torch.float16:
                tol = tol + 2.0 ** -25 * v.abs().sum(0).repeat_interleave(g, 0)
            tol = tol + torch.finfo(out.dtype).eps / 2 * (want.abs() + tol) + 2.0 ** -25
            err = (got - want).abs()
            assert bool((err <= tol).all()), (b, i, float((err / tol).max()))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("q, ctx, bound", [([40, 3], [200, 200], 128), ([90, 70], [100, 300], 64), ([3, 2], [300, 31], 30),
                                           ([4, 1], [1000, 900], 900), ([130], [520], 400), ([20], [10], 5)])
def test_causal_mask_where_the_context_is_cut(dt, q, ctx, bound):
    c = Case(q, ctx, 16, 4, 128, 16, dt, seed=bound)
    c.max_ctx = bound
    for ws in (None, c.workspace()):
        check(c, c.run(True, ws), bound)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("q", [3, 100])
def test_causal_mask_where_the_table_ends(dt, q):
    """A context length far past the table's reach: every token sees all that the table holds."""
    c = Case([q, q], [128, 128], 16, 4, 64, 16, dt, seed=q)
    c.ctx_d.fill_(2 ** 31 - 1)
    c.max_ctx = 128
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), False)
    assert pa.pa_device_status() == 0
