"""pa_decode_weights keeps 24 bits of every softmax weight on its way to the outputs.

Queries have one dim that is not zero, so that a score is one product, exact in fp32; value t is 1 in dim t and zero
elsewhere, so that dim t of an output is the weight of token t alone.

Tolerance, with e = 2^-24 (half a step of fp32). Scores are at most 1, base 2 below 1.45: their factor (scale times
log2 of e) rounds once ahead and once as a product, the maximum alike, and their difference once more:
ln 2 (4 * 1.45 + 2.9) e < 7 e; exp2 is good to 2 units, 4 e. So a weight is off by less than 11 e of itself, the sum
under it by as much and by its own roundings, at most n / 16 + 8 <= 15 (n <= 100 tokens, partial sums over lanes and
warps); the merge of the warps multiplies and adds twice more (their factors are exp2: 4 e), the quotient rounds
twice. Together under 2 * 11 + 15 + 8 + 4 = 49 e for exact parts of the weights; the weights' parts in 16 bits may add
2 e (two of fp16: 11 bits and a sign each; three of bf16: none). The output rounds by half a step, e, and dims whose
value is zero stay zero."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, E, Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("hq,hkv,d,lens", [(16, 2, 64, (64, 33, 7)), (8, 8, 128, (100,) * 5), (40, 2, 128, (97, 64))])
def test_outputs_hold_24_bits_of_a_weight(dt, hq, hkv, d, lens):
    paged = Paged(lens, hkv, d, 16, dt, 21)
    g = torch.Generator(device="cuda").manual_seed(22)
    q = torch.zeros(len(lens), hq, d, dtype=DT[dt], device="cuda")
    q[:, :, 0] = 1
    want = torch.zeros(len(lens), hq, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        key = (torch.rand(n, hkv, generator=g, device="cuda") * 2 - 1).to(DT[dt])
        t = torch.arange(n, device="cuda")
        blk = torch.from_numpy(paged.table[b].astype("int64")).cuda()[t // paged.bs]
        paged.k[blk, t % paged.bs] = 0
        paged.k[blk, t % paged.bs, :, 0] = key
        paged.v[blk, t % paged.bs] = torch.eye(n, d, dtype=DT[dt], device="cuda")[:, None].expand(n, hkv, d)
        want[b, :, :n] = torch.softmax(key.double(), 0).T.repeat_interleave(hq // hkv, 0)
    out = torch.full((len(lens), hq, d), float("nan"), device="cuda")
    w = torch.zeros(len(lens), hkv, paged.max_ctx, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_size(len(lens), hq, hkv, d, 16, paged.max_ctx), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, paged.max_ctx, 1.0, ws)
    err = (out.double() - want).abs()
    assert bool((err <= 52 * E * want).all()), float((err / want.clamp(min=1e-30)).max() / E)


@pytest.mark.parametrize("dt", list(DT))
def test_outputs_are_not_cut_in_one_direction(dt):
    """Many positive values of one size: an output is off by roundings of either sign, whose mean over all outputs
    is near nothing, and by what the tensor cores cut off within one tile, 2 e a product at most and three of them a
    tile. (Cut at every tile of a context, 66 of them here, the loss would be ten times that.) Mean of the relative
    errors: 6 e, and 2 e for what is left of the roundings: a sum of 66 tiles rounds by less than sqrt(66) e in the
    root mean square, its mean over 2,048 rows by a 45th of that."""
    B, hq, hkv, d, n = 64, 32, 8, 128, 2100
    paged = Paged((n,) * B, hkv, d, 16, dt, 23)
    g = torch.Generator(device="cuda").manual_seed(24)
    q = torch.zeros(B, hq, d, dtype=DT[dt], device="cuda")
    q[:, :, 0] = 1
    paged.k.zero_()
    paged.k[..., 0] = (torch.rand(paged.k.shape[:3], generator=g, device="cuda") * 2 - 1).to(DT[dt])
    paged.v.copy_(torch.rand(paged.v.shape, generator=g, device="cuda") * 0.5 + 0.5)
    out = torch.empty(B, hq, d, device="cuda")
    w = torch.zeros(B, hkv, n, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_size(B, hq, hkv, d, 16, n), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, n, 1.0, ws)
    t = torch.arange(n, device="cuda")
    mean = 0.0
    for b in range(B):
        blk = torch.from_numpy(paged.table[b].astype("int64")).cuda()[t // 16]
        p = torch.softmax(paged.k[blk, t % 16, :, 0].double(), 0)
        want = torch.einsum("th,thd->hd", p, paged.v[blk, t % 16].double()).repeat_interleave(hq // hkv, 0)
        mean += float(((out[b].double() - want) / want).mean()) / B
    assert abs(mean) <= 8 * E, mean / E


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("hq,hkv,d,lens", [(16, 2, 64, (64, 33, 7)), (8, 8, 128, (100,) * 5), (40, 2, 128, (97, 64))])
def test_small_weights_keep_their_bits(dt, hq, hkv, d, lens):
    """The same with scores from -8 to 0: weights down to 2^-11.6 of the largest. Scores of 11.6 (base 2) round by
    ln 2 (4 + 1) 11.6 e < 41 e, exp2 by 4: in place of 49 e, 2 * 45 + 15 + 8 + 4 = 117 e. fp16's parts end 2^-32 below the
    largest weight (2^-25 of numbers that are raised by 2^7), half a step of that for each of two."""
    paged = Paged(lens, hkv, d, 16, dt, 25)
    g = torch.Generator(device="cuda").manual_seed(26)
    q = torch.zeros(len(lens), hq, d, dtype=DT[dt], device="cuda")
    q[:, :, 0] = 1
    want = torch.zeros(len(lens), hq, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        key = (torch.rand(n, hkv, generator=g, device="cuda") * -8).to(DT[dt])
        key[n // 2] = 0
        t = torch.arange(n, device="cuda")
        blk = torch.from_numpy(paged.table[b].astype("int64")).cuda()[t // paged.bs]
        paged.k[blk, t % paged.bs] = 0
        paged.k[blk, t % paged.bs, :, 0] = key
        paged.v[blk, t % paged.bs] = torch.eye(n, d, dtype=DT[dt], device="cuda")[:, None].expand(n, hkv, d)
        want[b, :, :n] = torch.softmax(key.double(), 0).T.repeat_interleave(hq // hkv, 0)
    out = torch.full((len(lens), hq, d), float("nan"), device="cuda")
    w = torch.zeros(len(lens), hkv, paged.max_ctx, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_size(len(lens), hq, hkv, d, 16, paged.max_ctx), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, paged.max_ctx, 1.0, ws)
    err = (out.double() - want).abs()
    assert bool((err <= 120 * E * want + (2.0 ** -32 if dt == "fp16" else 0.0)).all()), float((err / want.clamp(min=1e-30)).max() / E)


@pytest.mark.parametrize("run", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (16, 1, 128)])
def test_fp16_scores_that_rise_by_single_steps(hq, hkv, d, run):
    """Scores of 2^27 (base 2) and more, where fp32's steps are 16, rising by a step or two every `run` tokens: a
    running maximum that is not moved for so little, because 8 more than it rounds to the same, makes weights of 2^16,
    which fp16 does not hold. Raw scores are 2^30 + 128 t, exact; a step is 23 (base 2), rounded to 16 or 32, so that
    all but the last run weigh 2^-16 of it at most and half as much again each run before: in all, of 12 equal runs,
    below 2^-15, and an output is the mean of the last run's values within 2^-14 of the largest one."""
    n = 12 * run
    paged = Paged((n,), hkv, d, 16, "fp16", 27)
    t = torch.arange(n, device="cuda")
    blk = torch.from_numpy(paged.table[0].astype("int64")).cuda()[t // 16]
    q = torch.zeros(1, hq, d, dtype=torch.float16, device="cuda")
    q[:, :, 0], q[:, :, 1] = 2.0 ** 15, 1
    paged.k[blk, t % 16] = 0
    paged.k[blk, t % 16, :, 0] = 2.0 ** 15
    paged.k[blk, t % 16, :, 1] = (128.0 * (t // run)).half()[:, None].expand(n, hkv)
    out = torch.empty(1, hq, d, device="cuda")
    w = torch.zeros(1, hkv, n, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_size(1, hq, hkv, d, 16, n), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, n, 2.0 ** -3, ws)
    v = paged.seq_v[0].double()
    want = v[-run:].mean(0).repeat_interleave(hq // hkv, 0)
    assert bool(((out[0].double() - want).abs() <= 2.0 ** -14 * v.abs().max()).all())
    share = w[0].double() / (hq // hkv)
    assert bool(((share[:, -run:] - 1 / run).abs() <= 2.0 ** -14 / run).all()) and bool((share[:, :-run] <= 2.0 ** -15 / run).all())
