"""One eviction of several sequences whose blocks come from the block manager's group compaction: every kept row, of
every sequence, is the one that lay there before, in a pool with next to no blocks to spare; and decode goes on."""
import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, i32, kept_by

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("lens,keep", [((300, 41, 500, 129), 64), ((900, 900, 17, 900, 33, 640), 256), ((16,) * 9, 16)])
def test_rows_of_a_group(dt, lens, keep):
    hkv, d, bs = 3, 64, 16
    seqs = list(range(len(lens)))
    new_lens = [min(keep, n) for n in lens]
    blocks = sum(-(-n // bs) for n in lens) + sum(-(-n // bs) for n in new_lens) + 2
    rng = np.random.default_rng(3)
    bm = pa.BlockManager(blocks, bs, free_order=rng.permutation(blocks))
    for s, n in zip(seqs, lens):
        bm.allocate(s, n)
    bm.fork(0, 50)                                  # keeps its blocks
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(blocks, bs, hkv, d, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    longest = max(lens)
    w = torch.rand(len(lens), hkv, longest, generator=g, device="cuda")

    def rows(cache, table, n):
        at = torch.arange(n, device="cuda")
        return cache[torch.tensor(table, device="cuda")[at // bs], at % bs].clone()

    def padded(tables):
        width = max(len(t) for t in tables)
        return i32([t + [0] * (width - len(t)) for t in tables])

    old = [bm.block_table(s) for s in seqs]
    before = [(rows(k, t, n), rows(v, t, n)) for t, n in zip(old, lens)]
    new = bm.compact_group(seqs, new_lens)
    kept = torch.full((len(lens), hkv, keep), -1, dtype=torch.int32, device="cuda")
    nw = torch.full((len(lens), hkv, keep), -1.0, device="cuda")
    pa.pa_evict(kept, nw, w, k, v, padded(old), i32(lens), padded(new), i32([keep] * len(lens)), longest, sinks=2, recent=8)
    for b, n in enumerate(lens):
        for h in range(hkv):
            want = kept_by(w[b, h].cpu().double().numpy(), n, keep, 2, 8)
            assert kept[b, h, :new_lens[b]].tolist() == want
            assert torch.equal(rows(k, new[b], new_lens[b])[:, h], before[b][0][want, h])
            assert torch.equal(rows(v, new[b], new_lens[b])[:, h], before[b][1][want, h])
    assert torch.equal(rows(k, bm.block_table(50), lens[0]), before[0][0])
    q = torch.randn(len(lens), hkv, d, generator=g, device="cuda").to(DT[dt])
    out = torch.empty(len(lens), hkv, d, device="cuda")
    pa.pa_decode(out, q, k, v, padded([bm.block_table(s) for s in seqs]), i32(new_lens), max(new_lens), d ** -0.5)
    for b, n in enumerate(new_lens):
        for h in range(hkv):
            kk, vv = rows(k, new[b], n)[:, h].double(), rows(v, new[b], n)[:, h].double()
            want = torch.softmax(q[b, h].double() @ kk.T * d ** -0.5, -1) @ vv
            assert float((out[b, h].double() - want).abs().max()) <= 2e-3
