"""pa_evict against a sort in plain Python: positions, weights and moved rows, all exact; and the whole path:
rotate and append, attend with weights, evict, attend again."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, Paged, check_weights, i32, kept_by, weights_after

pytestmark = pytest.mark.gpu


def evict(paged, w, keep, sinks, recent, most=None, max_ctx=None):
    """Run the eviction into fresh blocks behind the pool's; returns (kept, new weights, k, v, new table)."""
    B, bs = len(paged.lens), paged.bs
    new = [max(0, min(k, n)) for k, n in zip(keep, paged.lens)]
    need = [-(-n // bs) for n in new]
    perm = paged.blocks + np.random.default_rng(1).permutation(sum(need) + 2)
    table = np.full((B, max(1, max(need))), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    grow = torch.zeros(sum(need) + 2, *paged.k.shape[1:], dtype=paged.k.dtype, device="cuda")
    k, v = torch.cat([paged.k, grow + 5]), torch.cat([paged.v, grow + 6])
    most = most or max(1, max(new))
    kept = torch.full((B, paged.hkv, most), -7, dtype=torch.int32, device="cuda")
    nw = torch.full((B, paged.hkv, most + 2), -7.0, device="cuda")
    pa.pa_evict(kept, nw, w, k, v, paged.tables, paged.context_lens, i32(table), i32(keep), max_ctx or paged.max_ctx,
                sinks=sinks, recent=recent)
    return kept, nw, k, v, table


def check(paged, w, keep, sinks, recent, got):
    kept, nw, k, v, table = got
    host, bs = w.cpu().double().numpy(), paged.bs
    untouched = torch.ones(k.shape[:3], dtype=torch.bool, device="cuda")
    for b, n in enumerate(paged.lens):
        if keep[b] < 0:
            assert bool((kept[b] == -7).all()) and bool((nw[b] == -7).all())
            continue
        new = min(keep[b], n)
        assert bool((kept[b, :, new:] == -7).all()) and bool((nw[b, :, new:] == -7).all())
        at = torch.arange(new, device="cuda")
        blk = torch.from_numpy(table[b].astype(np.int64)).cuda()[at // bs] if new else at
        for h in range(paged.hkv):
            want = torch.tensor(kept_by(host[b, h], n, keep[b], sinks, recent), device="cuda")
            assert kept[b, h, :new].tolist() == want.tolist(), (b, h)
            if new == 0:
                continue
            assert torch.equal(nw[b, h, :new].nan_to_num(-3.0), w[b, h][want].nan_to_num(-3.0))
            assert torch.equal(k[blk, at % bs, h], paged.seq_k[b][want, h])
            assert torch.equal(v[blk, at % bs, h], paged.seq_v[b][want, h])
            untouched[blk, at % bs, h] = False
    old = paged.blocks
    assert torch.equal(k[:old].nan_to_num(9), paged.k.nan_to_num(9)) and torch.equal(v[:old].nan_to_num(9), paged.v.nan_to_num(9))
    assert bool((k[old:][untouched[old:]] == 5).all()) and bool((v[old:][untouched[old:]] == 6).all())


def table_of(kind, B, hkv, n, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.rand(B, hkv, n, generator=g, device="cuda").pow_(6)
    if kind == "ties":
        w = (w * 8).floor()
    elif kind == "equal":
        w.fill_(0.25)
    elif kind == "signs":
        w = torch.randn(B, hkv, n, generator=g, device="cuda")
        w = torch.where(w.abs() < 0.3, torch.where(w < 0, -0.0, 0.0), w)
    elif kind == "special":
        w = torch.randn(B, hkv, n, generator=g, device="cuda")
        pick = torch.rand(B, hkv, n, generator=g, device="cuda")
        for lo, val in ((0.0, math.nan), (0.1, math.inf), (0.15, -math.inf), (0.2, 1e-42), (0.25, 3.4e38)):
            w[(pick >= lo) & (pick < lo + 0.05)] = val
    return w


SHAPES = [  # lens, keep, sinks, recent, hkv, d, block size
    ((1,), (1,), 0, 0, 1, 64, 16), ((50, 9, 0, 33), (20, 20, 5, 33), 4, 8, 2, 64, 16), ((300, 257), (16, 0), 4, 16, 3, 128, 16),
    ((90, 90, 90), (40, -1, 1), 3, 50, 4, 64, 8), ((1000, 1025), (999, 512), 0, 0, 8, 128, 32), ((64,), (10,), 20, 4, 2, 64, 1),
    ((2049, 100), (300, 99), 1, 0, 2, 64, 7), ((5000,), (4097,), 4, 64, 2, 128, 256), ((800,), (700,), 0, 699, 18, 64, 16),
]


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "signs", "special"])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_a_sort(shape, kind):
    lens, keep, sinks, recent, hkv, d, bs = shape
    paged = Paged(lens, hkv, d, bs, "bf16", 1)
    w = table_of(kind, len(lens), hkv, paged.max_ctx + 1)
    check(paged, w, keep, sinks, recent, evict(paged, w, keep, sinks, recent))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("d", [8, 64, 96, 128, 256])
def test_every_type_and_head_dim(dt, d):
    paged = Paged((200, 31), 3, d, 16, dt, 2)
    w = table_of("random", 2, 3, 200)
    check(paged, w, (77, 30), 2, 9, evict(paged, w, (77, 30), 2, 9))


@pytest.mark.parametrize("kind", ["random", "ties", "equal"])
@pytest.mark.parametrize("n,keep", [(8200, 3000), (32768, 4096), (32769, 100), (70001, 33333)])
def test_long_contexts(kind, n, keep):
    paged = Paged((n, 50), 1, 64, 16, "fp16", 3)
    w = table_of(kind, 2, 1, n)
    check(paged, w, (keep, 20), 4, 32, evict(paged, w, (keep, 20), 4, 32))


def test_longer_keeps_are_cut_and_foreign_blocks_are_not_moved():
    paged = Paged((100,), 2, 64, 16, "bf16", 4)
    w = table_of("random", 1, 2, 100)
    kept, nw, k, v, table = evict(paged, w, (60,), 0, 0, most=40)          # kept holds 40
    for h in range(2):
        assert kept[0, h].tolist() == kept_by(w[0, h].cpu().double().numpy(), 100, 40, 0, 0)
    k0 = k.clone()
    bad = torch.tensor(table).cuda()
    bad[0, 1] = -4
    old = paged.tables.clone()
    old[0, 0] = 1 << 29
    kept2, nw2 = torch.zeros_like(kept), torch.zeros_like(nw)
    k[paged.blocks:] = 8
    pa.pa_evict(kept2, nw2, w, k, v, old, paged.context_lens, bad, i32([40]), 100)
    assert torch.equal(kept2, kept)
    t0 = int(table[0, 0])
    for j in range(16):
        for h in range(2):
            same = torch.equal(k[t0, j, h], k0[t0, j, h])
            assert same if int(kept[0, h, j]) >= 16 else bool((k[t0, j, h] == 8).all())
    assert bool((k[int(table[0, 1])] == 8).all())


def test_captured_and_replayed():
    paged = Paged((700, 90), 4, 128, 16, "bf16", 5)
    w = table_of("random", 2, 4, 700)
    want = evict(paged, w, (300, 80), 4, 32)
    k, v = want[2].clone(), want[3].clone()
    k[paged.blocks:], v[paged.blocks:] = 5, 6
    kept, nw, table, keep = torch.full_like(want[0], -7), torch.full_like(want[1], -7.0), i32(want[4]), i32([300, 80])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_evict(kept, nw, w, k, v, paged.tables, paged.context_lens, table, keep, 700, sinks=4, recent=32)
    for _ in range(2):
        graph.replay()
        assert torch.equal(kept, want[0]) and torch.equal(nw, want[1])
        assert torch.equal(k.nan_to_num(9), want[2].nan_to_num(9)) and torch.equal(v.nan_to_num(9), want[3].nan_to_num(9))


def test_a_bounded_cache_end_to_end():
    """A prompt normed, rotated and appended, its weights from the last queries, decode steps that add theirs,
    the eviction through the block manager (a forked sequence keeps its own blocks), and a decode over what is
    left: each against 64-bit operations on what the step before left."""
    H, hkv, D, bs, n, steps, keep = 8, 2, 64, 16, 150, 5, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    total = n + steps
    qkv = torch.randn(total, H + 2 * hkv, D, generator=g, device="cuda").bfloat16()
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2))
    f = torch.from_numpy(pa.pa_rope_frequencies(D, 1e4)[0]).cuda()
    bm = pa.BlockManager(64, bs)
    bm.allocate(0, n)
    k, v = (torch.full((64, bs, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = lambda: i32([bm.block_table(0) + [0] * (16 - len(bm.block_table(0)))])  # noqa: E731
    slots = pa.pa_compute_slot_mapping(table().cpu().numpy(), np.zeros(n, np.int32), np.arange(n, dtype=np.int32), bs)
    q = torch.empty(total, H, D, dtype=torch.bfloat16, device="cuda")

    def append(lo, hi, slots):
        r = qkv[lo:hi]
        pa.pa_norm_rope_and_cache(q[lo:hi], r[:, :H], r[:, H:H + hkv], r[:, H + hkv:], qw, kw, 1e-6, k, v,
                                  torch.as_tensor(slots, device="cuda"), torch.arange(lo, hi, dtype=torch.int32, device="cuda"), f)

    def rows(cache, count):
        t = torch.tensor(bm.block_table(0), device="cuda")
        at = torch.arange(count, device="cuda")
        return cache[t[at // bs], at % bs]

    class Seen:   # what weights_after needs of the cache as it stands
        pass

    def seen(count):
        s = Seen()
        s.lens, s.hkv, s.seq_k = [count], hkv, [rows(k, count)]
        return s

    scale = D ** -0.5
    append(0, n, slots)
    w = torch.full((1, hkv, 256), float("nan"), device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    old = w.clone()
    pa.pa_prefill_weights(w, q[:n], k, table(), i32([n]), i32([0, n]), n, n, scale, ws, window=32)
    check_weights(w, *weights_after(seen(n), old, [q[:n]], scale, 0.0, H, 32))
    out = torch.empty(1, H, D, dtype=torch.float32, device="cuda")
    for i in range(steps):
        slot, src, dst = bm.append_slot(0)
        assert src == -1
        append(n + i, n + i + 1, [slot])
        old = w.clone()
        pa.pa_decode_weights(out, w, q[n + i:n + i + 1], k, v, table(), i32([n + i + 1]), n + i + 1, scale, ws)
        check_weights(w, *weights_after(seen(n + i + 1), old, [q[n + i:n + i + 1]], scale, 1.0, H))
    bm.fork(0, 1)
    before_k, before_v, old_table = rows(k, total), rows(v, total), bm.block_table(0)
    new = bm.compact(0, keep)
    assert not set(new) & set(old_table) and bm.block_table(1) == old_table and bm.num_tokens(0) == keep
    kept = torch.empty(1, hkv, keep, dtype=torch.int32, device="cuda")
    nw = torch.empty(1, hkv, 256, device="cuda")
    pa.pa_evict(kept, nw, w, k, v, i32([old_table]), i32([total]), i32([new]), i32([keep]), total, sinks=2, recent=8)
    for h in range(hkv):
        want = kept_by(w[0, h].cpu().double().numpy(), total, keep, 2, 8)
        assert kept[0, h].tolist() == want
        assert torch.equal(rows(k, keep)[:, h], before_k[want, h]) and torch.equal(rows(v, keep)[:, h], before_v[want, h])
    t1 = torch.tensor(bm.block_table(1), device="cuda")
    at = torch.arange(total, device="cuda")
    assert torch.equal(k[t1[at // bs], at % bs], before_k)     # the fork's blocks are as they were
    pa.pa_decode(out, q[-1:], k, v, table(), i32([keep]), keep, scale)
    g_ = H // hkv
    for h in range(H):
        kk, vv = rows(k, keep)[:, h // g_].double(), rows(v, keep)[:, h // g_].double()
        ref = torch.softmax(q[-1, h].double() @ kk.T * scale, -1) @ vv
        assert float((out[0, h].double() - ref).abs().max()) <= 2e-3
