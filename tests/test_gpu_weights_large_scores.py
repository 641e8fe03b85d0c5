"""Attention weights of rows whose scores are large, or whose scale is negative, zero or tiny.

Tied scores. Queries and keys are constant rows of powers of two times small whole numbers: every score is exact in
fp32, and differs from the next kind by far more than 2^-x can bridge. So a row's weight lies in equal parts on its
highest-scoring tokens. Tolerance, with e = 2^-24: the count of them is exact (below 2^24), its inverse rounds once
(e), 2^0 is exact, and R rows add up with R roundings at most, another few where partial sums are joined: (R + 8) e.

Sums. For scores of any values, a row's weights add up to 1 however large the scores are, because numerators and the
sum under them come from the same differences: exp2 is good to 4 e on either side, a numerator's difference from the
row's maximum rounds once on its way (x e with x 2^-x below 0.54), and where the running maximum moves the sum is
multiplied by another exp2: 5 e each, at most once for every 32 of n keys. Sums of n terms round n / 16 + 32 times at
most. So (n / 4 + 64) e for a row, R e more for the sum over R rows, and as much again for adding the n results."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, E, Paged, check_weights, i32, weights_after

pytestmark = pytest.mark.gpu

SHAPES = [  # query lengths, context lengths, hq, hkv, d, block size, window
    ([3, 1], [700, 460], 16, 4, 64, 16, 0),            # few rows: they are held in both passes
    ([5, 40], [5, 1000], 8, 2, 128, 32, 8),
    ([150, 37], [800, 37], 8, 2, 128, 64, 0),          # more rows than a tile
    ([150, 20], [450, 20], 12, 4, 64, 7, 0),           # no power of two: rows are gathered
    ([900], [3000], 16, 4, 128, 16, 0),                # rows in pieces
]


def call(paged, q, start, scale, window):
    B, n = len(start) - 1, max(b - a for a, b in zip(start, start[1:]))
    w = torch.zeros(B, paged.hkv, paged.max_ctx + 1, device="cuda")
    size = pa.pa_prefill_weights_workspace_size(B, q.shape[0], q.shape[1], paged.hkv, paged.d, paged.bs, n, paged.max_ctx, window)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    pa.pa_prefill_weights(w, q, paged.k, paged.tables, paged.context_lens, i32(start), n, paged.max_ctx, scale, ws, window=window)
    return w


def starts(qlens):
    start = [0]
    for n in qlens:
        start.append(start[-1] + n)
    return start


def fill_keys(paged, b, keys):
    """Keys [n, Hkv, D] of sequence b, written to its blocks."""
    n = keys.shape[0]
    t = torch.arange(n, device="cuda")
    blk = torch.from_numpy(paged.table[b].astype("int64")).cuda()[t // paged.bs]
    paged.k[blk, t % paged.bs] = keys
    paged.seq_k[b] = keys


def check_tied(shape, dt, a, b, sign, spread):
    qlens, lens, hq, hkv, d, bs, window = shape
    paged = Paged(lens, hkv, d, bs, dt, 7)
    for i, n in enumerate(lens):   # keys b, 2 b or 3 b (or all alike), runs of 150 tokens
        level = 1 + (torch.arange(n, device="cuda") // 150) % 3 if spread else torch.ones(n, device="cuda")
        fill_keys(paged, i, (b * level.double()).to(DT[dt])[:, None, None].expand(n, hkv, d))
    start = starts(qlens)
    q = torch.full((start[-1], hq, d), a, dtype=DT[dt], device="cuda")
    w = call(paged, q, start, 2.0 ** -3 * sign, window).double()
    g = hq // hkv
    for i, (n, ctx) in enumerate(zip(qlens, lens)):
        count = min(n, window) if window else n
        keys = paged.seq_k[i][:, 0, 0].double() * sign
        j = torch.arange(ctx, device="cuda")
        sees = j[None] < ctx - count + 1 + torch.arange(count, device="cuda")[:, None]
        s = keys[None].expand(count, ctx).masked_fill(~sees, -torch.inf)
        best = (s == s.amax(-1, keepdim=True)) & sees
        want = (best.double() / best.sum(-1, keepdim=True)).sum(0) * g
        err = (w[i, :, :ctx] - want).abs()
        assert bool((err <= (count * g + 8) * E * want).all()), (i, float((err / want.clamp(min=1e-9)).max()))
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("log2", [20, 26, 28, 33, 64, 118])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_tied_scores_bf16_and_fp32(shape, log2, sign, spread):
    """Scores of about 2^log2 (times head_dim / 8), of one sign or the other."""
    for dt in ("bf16", "fp32"):
        check_tied(SHAPES[shape], dt, 2.0 ** (log2 // 2), 2.0 ** (log2 - log2 // 2), sign, spread)


@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("log2", [20, 26, 29])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_tied_scores_fp16(shape, log2, sign, spread):
    check_tied(SHAPES[shape], "fp16", 2.0 ** 15, 2.0 ** (log2 - 15), sign, spread)


@pytest.mark.parametrize("scale", [0.125, -0.09])
@pytest.mark.parametrize("log2", [0, 12, 16, 20, 24, 28, 60, 100])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_rows_add_up_to_one(shape, log2, scale):
    """Random scores of about 2^log2 times the root of head_dim: a row's weights add up to 1."""
    qlens, lens, hq, hkv, d, bs, window = SHAPES[shape]
    for dt in DT:
        if dt == "fp16" and log2 > 24:
            continue
        paged = Paged(lens, hkv, d, bs, dt, 11, by=2.0 ** (log2 // 2))
        start = starts(qlens)
        gen = torch.Generator(device="cuda").manual_seed(12)
        q = (torch.randn(start[-1], hq, d, generator=gen, device="cuda") * 2.0 ** (log2 - log2 // 2)).to(DT[dt])
        w = call(paged, q, start, scale, window).double()
        for i, (n, ctx) in enumerate(zip(qlens, lens)):
            rows = (min(n, window) if window else n) * (hq // hkv)
            off = (w[i, :, :ctx].sum(-1) / rows - 1).abs()
            assert bool((off <= 2 * (ctx / 4 + 64 + rows) * E).all()), (dt, i, float(off.max()))
            # the last query token sees everything, the token before it all but one: no key past a row's reach weighs
            assert bool((w[i, :, :ctx] >= 0).all()) and bool((w[i, :, ctx:] == 0).all())


@pytest.mark.parametrize("scale", [-0.125, 0.0, 1e-42, -1e-42])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_negative_zero_and_tiny_scales(shape, dt, scale):
    qlens, lens, hq, hkv, d, bs, window = SHAPES[shape]
    paged = Paged(lens, hkv, d, bs, dt, 13)
    start = starts(qlens)
    gen = torch.Generator(device="cuda").manual_seed(14)
    q = (torch.randn(start[-1], hq, d, generator=gen, device="cuda") * 1.5).to(DT[dt])
    w = call(paged, q, start, scale, window)
    old = torch.zeros_like(w)
    check_weights(w, *weights_after(paged, old, [q[a:b] for a, b in zip(start, start[1:])], scale, 0.0, hq, window))


@pytest.mark.parametrize("scale", [-0.125, 0.0, 1e-42])
@pytest.mark.parametrize("dt", list(DT))
def test_leading_rows_that_see_nothing(dt, scale):
    """More query tokens than context: the first ones see nothing, whatever the scale's sign."""
    for qlens, lens, hq in (([30], [12], 8), ([200], [150], 8)):
        paged = Paged(lens, 2, 64, 16, dt, 15)
        gen = torch.Generator(device="cuda").manual_seed(16)
        q = torch.randn(qlens[0], hq, 64, generator=gen, device="cuda").to(DT[dt])
        w = call(paged, q, starts(qlens), scale, 0)
        check_weights(w, *weights_after(paged, torch.zeros_like(w), [q], scale, 0.0, hq))


@pytest.mark.parametrize("scale", [-0.125, 0.0, 1e-42])
@pytest.mark.parametrize("dt", list(DT))
def test_decode_step_of_those_scales(dt, scale):
    lens, hq, hkv, d = (700, 1, 33), 16, 2, 128
    paged = Paged(lens, hkv, d, 16, dt, 17)
    gen = torch.Generator(device="cuda").manual_seed(18)
    q = (torch.randn(len(lens), hq, d, generator=gen, device="cuda") * 1.5).to(DT[dt])
    w = torch.zeros(len(lens), hkv, 700, device="cuda")
    out = torch.empty(len(lens), hq, d, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_size(len(lens), hq, hkv, d, 16, 700), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, 700, scale, ws)
    check_weights(w, *weights_after(paged, torch.zeros_like(w), [x[None] for x in q], scale, 1.0, hq))
