"""The few-rows prefill kernel multiplies by the softmax's weights in two parts, a
16-bit one and its 16-bit remainder, as decode does: held here to that precision,
against 64 bits and against decode itself.

Tolerance of one element, A the softmax average of |v|: what two parts leave of a
weight, (eps / 2)^2 A of the 16-bit type (fp16: a remainder below 2^-14 is off by up
to 2^-25 whole, where the largest weight is at least 1: 2^-25 sum |v| / l, and l is
at least a tenth of the tokens here); the score, twice (D + 2) 2^-23 |scale| max sum
|q| |k|, small by a small scale; the sums in fp32, 2 (n + 16) 2^-23 A; the output in
fp32, 2^-24 |y|. One rounding of the weights alone would be off by about eps / 2 A /
sqrt(n), some ten times more than this at the lengths used."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from prefill_cases import Case

pytestmark = pytest.mark.gpu

SCALE = 0.004


def truth(c, causal):
    """(output in 64 bits, tolerance) of every token, [tokens, Hq, D]."""
    g, eps = c.hq // c.hkv, torch.finfo(c.dt).eps
    want = torch.zeros(c.tokens, c.hq, c.d, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for b in range(c.n):
        for i in range(c.q_lens[b]):
            sees = c.ctx_lens[b] - (c.q_lens[b] - i - 1 if causal else 0)
            if sees <= 0:
                continue
            at = int(c.start[b]) + i
            q = c.query[at].double().view(c.hkv, g, c.d)
            k, v = c.k[b][:sees].double(), c.v[b][:sees].double()
            s = torch.einsum("hgd,chd->hgc", q, k) * SCALE
            p = torch.softmax(s, -1)
            assert float((s.amax(-1) - s.amin(-1)).max()) < 2.3   # every weight at least a tenth of the largest
            want[at] = torch.einsum("hgc,chd->hgd", p, v).reshape(c.hq, c.d)
            avg = torch.einsum("hgc,chd->hgd", p, v.abs()).reshape(c.hq, c.d)
            size = torch.einsum("hgd,chd->hgc", q.abs(), k.abs()).amax(-1).reshape(c.hq, 1)
            t = ((eps / 2) ** 2 + 2 * (sees + 16) * 2.0 ** -23 + 2 * (c.d + 2) * 2.0 ** -23 * SCALE * size) * avg
            if c.dt == torch.float16:
                t = t + 2.0 ** -25 * 10 * v.abs().mean(0).repeat_interleave(g, 0)
            tol[at] = t + 2.0 ** -24 * (want[at].abs() + t)
    return want, tol


SHAPES = [   # query lengths, context lengths, Hq, Hkv, D, block size (0: contiguous)
    ([4] * 4, [33, 20, 17, 4], 32, 8, 128, 16),
    ([1, 2, 3], [64, 5, 40], 16, 16, 64, 0),
    ([4] * 16, [260] * 16, 32, 8, 128, 32),          # ranges cut inside sequences: pieces merged
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_weights_in_two_parts(shape, dt):
    q, ctx, hq, hkv, d, bs = SHAPES[shape]
    c = Case(q, ctx, hq, hkv, d, bs, dt, seed=80 + shape, scale=SCALE)
    for causal in ((True, False) if bs else (False,)):
        want, tol = truth(c, causal)
        out = c.run(causal, c.workspace(), out_dtype=torch.float32).double()
        err = (out - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_single_tokens_are_decode(dt):
    """One query token a sequence: the two entry points within each other's tolerance."""
    c = Case([1] * 6, [1, 17, 60, 33, 64, 5], 32, 8, 128, 16, dt, seed=90, scale=SCALE)
    want, tol = truth(c, True)
    out = c.run(True, c.workspace(), out_dtype=torch.float32)
    ref = torch.empty_like(out)
    pa.pa_decode(ref, c.query, c.kc, c.vc, c.tables_d, c.ctx_d, c.max_ctx, c.scale)
    for x in (out, ref):
        assert bool(((x.double() - want).abs() <= tol).all())
    assert bool(((out - ref).double().abs() <= 2 * tol).all())
