"""pa_decode_weights with large scores: equal keys share a row's weight, in weights and outputs, up to 2^118.

Scores are exact in fp32 and differ from the next kind by far more than the softmax can bridge (constant rows of powers
of two times small whole numbers). Tolerance, with e = 2^-24: equal weights are 1 / n, rounded once, summed over the
query heads of a KV head (R e); an output is their sum with V in fp32, (n / 16 + 64) e of the average of |v|."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, E, Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dt,log2", [("bf16", 20), ("bf16", 30), ("bf16", 64), ("bf16", 118), ("fp32", 28), ("fp32", 118),
                                     ("fp16", 20), ("fp16", 29)])
@pytest.mark.parametrize("lens,hq,hkv,d", [((700, 1, 460), 16, 4, 64), ((5000, 33), 40, 2, 128)])
def test_tied_scores(lens, hq, hkv, d, dt, log2, sign):
    paged = Paged(lens, hkv, d, 16, dt, 51)
    a = 2.0 ** (15 if dt == "fp16" else log2 // 2)
    b = 2.0 ** log2 / a
    q = torch.full((len(lens), hq, d), a, dtype=DT[dt], device="cuda")
    for i, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        blk = torch.from_numpy(paged.table[i].astype("int64")).cuda()[t // 16]
        paged.seq_k[i] = ((1 + (t // 150) % 3).double() * b).to(DT[dt])[:, None, None].expand(n, hkv, d)
        paged.k[blk, t % 16] = paged.seq_k[i]
    out = torch.empty(len(lens), hq, d, device="cuda")
    w = torch.zeros(len(lens), hkv, paged.max_ctx, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_size(len(lens), hq, hkv, d, 16, paged.max_ctx), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, paged.max_ctx, 2.0 ** -3 * sign, ws)
    group = hq // hkv
    for i, n in enumerate(lens):
        keys = paged.seq_k[i][:, 0, 0].double() * sign
        best = keys == keys.max()
        want = best.double() / best.sum() * group
        assert bool(((w[i, :, :n].double() - want).abs() <= (group + 4) * E * want).all())
        v = paged.seq_v[i][best].double()
        mean, size = (x.mean(0).repeat_interleave(group, 0) for x in (v, v.abs()))
        assert bool(((out[i].double() - mean).abs() <= (n / 16 + 64) * E * size).all())
