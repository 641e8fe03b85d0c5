"""pa_prefill and pa_cross_attention against softmax attention in 64 bits, at
the sizes and masks where they can go wrong; tolerances as derived in
prefill_cases. What no sequence owns (cache tails, table tails, unused blocks)
holds NaN or ids outside the pool."""
import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from prefill_cases import Case

pytestmark = pytest.mark.gpu

LENS = {   # query lengths, context lengths
    "one": ([1], [1]),
    "prompts": ([25, 47, 12], [25, 47, 12]),
    "chunks": ([1, 7, 33, 64, 130, 0, 257], [129, 7, 500, 64, 1030, 40, 300]),
    "verify": ([4] * 5, [700, 33, 4, 128, 1000]),
    "empty rows": ([5, 9, 3, 2], [2, 0, 3, 1]),       # a query longer than its context: leading rows see nothing
    "tile edges": ([128, 127, 129, 32, 31], [128, 255, 257, 384, 31]),
}


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dims", [(4, 4, 64, 16), (8, 2, 128, 16)])
def test_paged(dt, causal, lens, dims):
    hq, hkv, d, bs = dims
    c = Case(*LENS[lens], hq, hkv, d, bs, dt, seed=len(lens))
    for ws in (None, c.workspace()):
        c.check(c.run(causal, ws), causal)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("bs", [1, 2, 4, 8, 12, 32, 64, 128, 256, 255])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_block_sizes(bs, dt):
    c = Case([40, 3, 200], [41, 300, 777], 8, 2, 128, bs, dt, seed=bs)
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), True)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (6, 1), (12, 2), (16, 1), (32, 2), (33, 1), (64, 1), (130, 1), (200, 1), (5, 5)])
@pytest.mark.parametrize("dt", ["fp16", "fp32"])
@pytest.mark.parametrize("q", [1, 50])
def test_head_layouts(hq, hkv, dt, q):
    c = Case([q, max(1, q // 3), q + 1], [q + 100, q, 333], hq, hkv, 64, 16, dt, seed=hq)
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), True)


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dims", [(16, 16, 64), (8, 2, 128)])
@pytest.mark.parametrize("lens", [([1, 1, 1], [1500, 1, 0]), ([44, 1, 300, 0, 7], [150, 1500, 129, 20, 64]),
                                  ([448, 300], [1500, 1500])])
def test_cross(dt, dims, lens):
    hq, hkv, d = dims
    c = Case(*lens, hq, hkv, d, 0, dt, seed=3, max_states=1511)
    for ws in (None, c.workspace()):
        c.check(c.run(False, ws), False)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_output_types(out_dtype, dt):
    c = Case([3, 70], [500, 70], 8, 2, 128, 16, dt, seed=8)
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws, out_dtype=out_dtype), True)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("q", [2, 90])
def test_rows_outside_every_sequence_are_left(dt, q):
    c = Case([q, 0, q], [q + 300, 50, q], 8, 2, 128, 16, dt, seed=9, lead=3, trail=37)
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), True)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_scales(scale, dt):
    """Zero (plain averages), negative, and peaked (the running maximum moves)."""
    c = Case([5, 100], [400, 300], 4, 2, 64, 16, dt, seed=10, scale=scale)
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), True)


def test_scores_that_climb():
    """Scores rising along the context by far more than the rescale's headroom: every tile moves the maximum."""
    for dt in ("bf16", "fp16", "fp32"):
        c = Case([64, 3], [900, 1000], 4, 1, 128, 16, dt, seed=11)
        for b in range(2):
            n = c.ctx_lens[b]
            c.k[b].mul_((torch.arange(n, device="cuda") / n * 6)[:, None, None].to(c.dt))
            flat = torch.full((-(-n // 16) * 16, 1, 128), float("nan"), dtype=c.dt, device="cuda")
            flat[:n] = c.k[b]
            c.kc[c.tables_d[b, :-(-n // 16)].long()] = flat.view(-1, 16, 1, 128)
        for ws in (None, c.workspace()):
            c.check(c.run(True, ws), True)


def test_bad_pages_read_as_zeros():
    """Table entries outside the pool, inside the context: their tokens are zero keys and values."""
    for dt in ("bf16", "fp32"):
        c = Case([40], [200], 4, 2, 128, 16, dt, seed=12)
        for page, bad in ((3, -1), (7, 10 ** 6)):
            c.tables_d[0, page] = bad
            c.k[0][page * 16:page * 16 + 16] = 0
            c.v[0][page * 16:page * 16 + 16] = 0
        for ws in (None, c.workspace()):
            c.check(c.run(True, ws), True)


def test_lengths_past_the_bounds_are_cut():
    """A context length above max_context_len or the table's reach is attended up to it; sequences whose
    query_start runs past the tokens, or backwards, write nothing out of range."""
    for dt in ("bf16", "fp32"):
        c = Case([4, 6], [64, 48], 4, 2, 128, 16, dt, seed=13)
        full = c.run(False, None)
        c.ctx_d.fill_(10 ** 9)
        c.max_ctx = 48
        out = c.run(False, None)
        assert torch.equal(out[4:], full[4:])
        c.start_d.copy_(torch.tensor([0, 10 ** 9, 3], dtype=torch.int32))
        big = torch.full((64, 4, 128), 5.0, dtype=c.dt, device="cuda")
        c.run(False, None, out=big[:10])
        torch.cuda.synchronize()
        assert bool((big[10:] == 5.0).all())
    assert pa.pa_device_status() == 0


def test_query_start_that_overlaps_stays_in_bounds():
    """Sequences that claim the same tokens again and again: more units than the batch's tokens can hold. The
    result is unspecified; nothing outside out and the workspace is written."""
    for hkv, q in ((2, 60), (2, 200), (4, 3)):
        c = Case([q] + [0] * 79, [700] * 80, 4 * hkv, hkv, 64, 16, "bf16", seed=13)
        starts = np.zeros(81, np.int32)
        starts[1::2] = q
        c.start_d.copy_(torch.from_numpy(starts))
        need = c.workspace().numel()
        big = torch.full((need + (32 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        out = torch.full((q + 64, 4 * hkv, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        c.run(True, big[:need], out=out[:q])
        torch.cuda.synchronize()
        assert bool((big[need:] == 0x5A).all()) and bool((out[q:] == 5.0).all())
    assert pa.pa_device_status() == 0


def test_single_tokens_agree_with_decode():
    """Query lengths of one: pa_decode's result."""
    c = Case([1] * 6, [1, 17, 300, 1029, 64, 555], 32, 8, 128, 16, "bf16", seed=14)
    out = c.run(True, c.workspace(), out_dtype=torch.float32)
    ref = torch.empty_like(out)
    pa.pa_decode(ref, c.query, c.kc, c.vc, c.tables_d, c.ctx_d, c.max_ctx, c.scale)
    c.check(out, True)
    c.check(ref, True)


def test_large_ragged_batch():
    rng = np.random.default_rng(15)
    q = rng.integers(0, 90, 150)
    ctx = q + rng.integers(0, 700, 150)
    for dt in ("bf16", "fp16"):
        c = Case(q.tolist(), ctx.tolist(), 8, 2, 64, 32, dt, seed=16)
        for ws in (None, c.workspace()):
            c.check(c.run(True, ws), True)


FEW = [   # query lengths, context lengths, Hq, Hkv, D, block size (0: contiguous)
    ([1], [1], 8, 8, 64, 16), ([4] * 16, [4164 - 3 * i for i in range(16)], 32, 8, 128, 16),
    ([3, 0, 1, 2, 0, 3], [3, 9, 0, 1, 40, 700], 20, 4, 128, 32), ([2, 1, 2], [1, 0, 2], 32, 8, 64, 64),
    ([16, 1, 7], [300, 15, 17], 6, 6, 128, 256), ([1] * 70, [(37 * i) % 900 for i in range(70)], 16, 16, 64, 0),
    ([4, 2], [1500, 31], 16, 4, 64, 0), ([2] * 200, [(71 * i) % 333 for i in range(200)], 40, 5, 64, 16),
    ([1, 1], [16, 65536], 32, 8, 128, 16),
]


@pytest.mark.parametrize("case", range(len(FEW)))
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_few_rows(case, dt):
    """At most 16 rows a KV head: with a workspace the ranges are cut between CTAs, pieces of a sequence joined;
    causal rows that see nothing of a piece; empty sequences and contexts."""
    q, ctx, hq, hkv, d, bs = FEW[case]
    c = Case(q, ctx, hq, hkv, d, bs, dt, seed=40 + case, lead=2, trail=3)
    for causal in ((True, False) if bs else (False,)):
        ws = c.workspace()
        out = c.run(causal, ws)
        c.check(out, causal)
        assert torch.equal(c.run(causal, c.workspace(fill=0)), out)
        c.check(c.run(causal, None), causal)
        c.check(c.run(causal, ws, out_dtype=torch.float32), causal)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("shape", [(186, 1, 700, 4, 8, 64, 128), (77, 4, 2000, 4, 4, 128, 128), (300, 2, 200, 2, 4, 64, 16),
                                   (95, 30, 2000, 1, 2, 128, 64)])
def test_many_short_pieces_a_cta(shape):
    """Far more sequences than CTAs, each of a few tiles: a CTA's producers run segments ahead of its products.
    The same bits every time."""
    n, q_hi, past, hkv, g, d, bs = shape
    rng = np.random.default_rng(n)
    q = rng.integers(0, q_hi + 1, n)
    q[0] = q_hi
    ctx = q + rng.integers(0, past + 1, n)
    for dt in ("fp16", "bf16"):
        c = Case(q.tolist(), ctx.tolist(), hkv * g, hkv, d, bs, dt, seed=24)
        for causal in (True, False):
            for ws in (None, c.workspace()):
                out = c.run(causal, ws)
                c.check(out, causal)
                for _ in range(10):
                    assert torch.equal(c.run(causal, ws), out)
    assert pa.pa_device_status() == 0


def test_long_prompt_and_long_context():
    """Many tiles per CTA, the whole pipeline's depth; 65,536 tokens of context."""
    c = Case([2000, 1], [2000, 2000], 8, 1, 128, 16, "bf16", seed=17)
    c.check(c.run(True, c.workspace()), True)
    c = Case([1, 130], [65536, 30000], 8, 1, 128, 16, "bf16", seed=18)
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), True)


def test_far_cache_offsets():
    """Used blocks whose byte offset passes 2^32."""
    c = Case([6, 40], [500, 100], 8, 2, 128, 16, "bf16", seed=19)
    rows = (1 << 32) // (16 * 2 * 128 * 2) + 64
    far = [torch.zeros(rows, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    n = c.kc.shape[0]
    far[0][-n:], far[1][-n:] = c.kc, c.vc
    want = c.run(True, c.workspace())
    c.kc, c.vc = far
    c.tables_d = torch.where((c.tables_d >= 0) & (c.tables_d < n), c.tables_d + (rows - n), c.tables_d)
    got = c.run(True, c.workspace())
    assert torch.equal(got, want)
    c.check(got, True)


def test_results_do_not_depend_on_the_run():
    """Bit for bit the same again, from a workspace holding anything, on another stream, captured and replayed with
    new inputs; two streams with their own workspaces at once."""
    cases = [Case([4] * 16, [900 + 10 * i for i in range(16)], 32, 8, 128, 16, "bf16", seed=20),
             Case([300, 20], [800, 1500], 16, 4, 128, 32, "fp16", seed=21)]
    wss = [c.workspace() for c in cases]
    want = [c.run(True, ws) for c, ws in zip(cases, wss)]
    for c, w in zip(cases, want):
        c.check(w, True)
        assert torch.equal(c.run(True, c.workspace(fill=0x3C)), w)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [torch.full_like(w, 5.0) for w in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, ws, o, s in zip(cases, wss, outs, streams):
            c.run(True, ws, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for c, ws, w in zip(cases, wss, want):
        q = c.query.clone()
        c.query.zero_()
        out = torch.full_like(w, 5.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(True, ws, out=out)
        c.query.copy_(q)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert pa.pa_device_status() == 0


def test_prompt_then_steps_then_cross():
    """As they would be used: prompts rotated into the cache and attended in two chunks, then decode steps
    (rotate, append, decode), each against dense attention over the rotated rows; then cross attention."""
    hq, hkv, d, bs, B = 8, 2, 64, 16, 3
    lens, steps, first = [70, 33, 5], 4, 20
    gen = torch.Generator(device="cuda").manual_seed(22)
    total = [n + steps for n in lens]
    rows = [torch.randn(t, hq + 2 * hkv, d, generator=gen, device="cuda").bfloat16() for t in total]
    f = torch.from_numpy(pa.pa_rope_frequencies(d, 1e4)[0]).cuda()
    bm = pa.BlockManager(64, bs)
    kc = torch.full((64, bs, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    for b in range(B):
        bm.allocate(b, lens[b])

    def tables():
        t = np.zeros((B, 8), np.int32)
        for b in range(B):
            ids = bm.block_table(b)
            t[b, :len(ids)] = ids
        return t

    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731

    def feed(ranges):
        """Append tokens ranges[b] = (from, to) of each sequence and attend them."""
        tab = tables()
        x = torch.cat([rows[b][lo:hi] for b, (lo, hi) in enumerate(ranges)])
        seq = np.concatenate([np.full(hi - lo, b) for b, (lo, hi) in enumerate(ranges)])
        pos = np.concatenate([np.arange(lo, hi) for lo, hi in ranges])
        slots = torch.from_numpy(pa.pa_compute_slot_mapping(tab, seq, pos, bs)).cuda()
        q = torch.empty(len(pos), hq, d, dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_and_cache(q, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, slots, i32(pos.tolist()), f)
        out = torch.empty(len(pos), hq, d, dtype=torch.float32, device="cuda")
        ctx = [hi for _, hi in ranges]
        starts = np.concatenate([[0], np.cumsum([hi - lo for lo, hi in ranges])]).tolist()
        if all(hi - lo == 1 for lo, hi in ranges):
            pa.pa_decode(out, q, kc, vc, i32(tab.tolist()), i32(ctx), max(ctx), d ** -0.5)
        else:
            pa.pa_prefill(out, q, kc, vc, i32(tab.tolist()), i32(ctx), i32(starts), max(hi - lo for lo, hi in ranges),
                          max(ctx), d ** -0.5)
        return [out[starts[b]:starts[b + 1]] for b in range(B)]

    got = [[] for _ in range(B)]
    plan = [[(0, min(first, n)) for n in lens], [(min(first, n), n) for n in lens]]
    for ranges in plan:
        for b, o in enumerate(feed(ranges)):
            got[b].append(o)
    for s in range(steps):
        for b in range(B):
            bm.append_slot(b)
        for b, o in enumerate(feed([(n + s, n + s + 1) for n in lens])):
            got[b].append(o)
    for b in range(B):
        n = total[b]
        x = rows[b].double().cpu()
        angle = torch.arange(n).double()[:, None] * f.cpu()[None]

        def turned(t):
            a, c = t[..., :d // 2], t[..., d // 2:]
            cs, sn = angle.cos()[:, None], angle.sin()[:, None]
            return torch.cat([a * cs - c * sn, c * cs + a * sn], -1)

        q, k, v = turned(x[:, :hq]), turned(x[:, hq:hq + hkv]), x[:, hq + hkv:]
        s = torch.einsum("nhgd,chd->hgnc", q.view(n, hkv, hq // hkv, d), k) * d ** -0.5
        s.masked_fill_(torch.ones(n, n).triu(1).bool(), -float("inf"))
        p = torch.softmax(s, -1)
        want = torch.einsum("hgnc,chd->nhgd", p, v).reshape(n, hq, d)
        avg = torch.einsum("hgnc,chd->nhgd", p, v.abs()).reshape(n, hq, d)
        size = torch.einsum("nhgd,chd->hgnc", q.view(n, hkv, hq // hkv, d).abs(), k.abs()).amax(-1)
        size = size.permute(2, 0, 1).reshape(n, hq, 1) * d ** -0.5
        # rotated queries and keys are rounded to bf16 (2^-8 each): scores off by 2^-7 of sum |q||k|, the
        # weights by as much, numerator and denominator; the weights themselves by 2^-8
        tol = (2 * 2.0 ** -7 * size + 2.0 ** -8 + 2.0 ** -12) * avg
        err = (torch.cat(got[b]).double().cpu() - want).abs()
        assert bool((err <= tol).all()), (b, float((err / tol).max()))
    # the decoder's queries over encoder states of another length
    c = Case([4, 1, 9], [40, 77, 13], hq, hkv, d, 0, "bf16", seed=23)
    c.check(c.run(False, c.workspace()), False)
    assert pa.pa_device_status() == 0


WAVES = [   # (query, context) lengths, Hq, Hkv, D, block size (0: contiguous), causal: how the last wave is given out
    ([256] * 5, [4096, 4000, 3000, 4096, 100], 8, 8, 64, 0, False),         # few units: cut into pieces, one a CTA
    ([256] * 9, [4096] * 9, 8, 8, 128, 0, False),                          # as many pieces as CTAs, nearly
    ([200] * 10, [7700 - 300 * i for i in range(10)], 8, 8, 64, 64, True),  # more units than half the CTAs: ranges
    ([100] * 4, [6200, 6100, 17, 6200], 8, 8, 64, 0, False),               # one row tile a unit
    ([100] * 10, [130 * 128] * 10, 8, 8, 64, 0, False),                    #   and ranges of them
    ([256] * 16, [1500] * 16, 8, 8, 64, 0, False),                         # short contexts: not cut
    ([60, 1, 300] * 11, [60, 700, 2000] * 11, 16, 8, 64, 32, True),        # drawn, longest contexts first
    ([12] * 300, [12 + (i * 7) % 90 for i in range(300)], 8, 8, 64, 16, True),     # more than are ordered
    ([12] * 256, [12 + (i * 7) % 90 for i in range(256)], 8, 8, 64, 16, True),     # as many
]


@pytest.mark.parametrize("i", range(len(WAVES)))
def test_last_wave_and_order(i):
    """However the units reach the CTAs: right, and the same bits on every run, from any workspace, in a graph."""
    q, ctx, hq, hkv, d, bs, causal = WAVES[i]
    c = Case(q, ctx, hq, hkv, d, bs, "bf16", seed=40 + i)
    ws = c.workspace()
    got = c.run(causal, ws)
    c.check(got, causal)
    assert torch.equal(c.run(causal, c.workspace(fill=0x11)), got)
    out = torch.full_like(got, 5.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(causal, ws, out=out)
        c.run(causal, ws, out=out)
    for _ in range(3):
        out.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("q, ctx", [([300, 7, 0, 130], [100, 700, 0, 1000]), ([2, 1, 3], [1, 900, 3]), ([70], [40])])
def test_loose_host_bounds(dt, q, ctx):
    """max_query_len and max_context_len are upper bounds: far larger ones (another kernel, other tiles, more
    workspace) give right results too, rows that see nothing among them."""
    c = Case(q, ctx, 8, 2, 128, 16, dt, seed=60)
    c.max_q, c.max_ctx = 5000, c.tables.shape[1] * 16
    for ws in (None, c.workspace()):
        c.check(c.run(True, ws), True)
    c = Case(q, ctx, 8, 2, 64, 0, dt, seed=61, max_states=3000)
    c.max_q, c.max_ctx = 1000, 3000
    for ws in (None, c.workspace()):
        c.check(c.run(False, ws), False)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q, ws", [(4, True), (100, False), (300, False), (300, True)])
def test_output_at_any_16_bytes(out_dtype, q, ws):
    """out is 16-byte aligned, no more; what lies beside it stays as it was."""
    c = Case([q, 1, q // 2], [q + 500, 1, q + 2000], 16, 4, 64, 16, "bf16", seed=70)
    ws = c.workspace() if ws else None
    want = c.run(True, ws, out_dtype=out_dtype)
    c.check(want, True)
    pad = 16 // want.element_size()
    flat = torch.full((want.numel() + 2 * pad + 64,), 5.0, dtype=out_dtype, device="cuda")
    out = flat[pad:pad + want.numel()].view(want.shape)
    assert out.data_ptr() % 32 == 16
    assert torch.equal(c.run(True, ws, out=out), want)
    assert bool((flat[:pad] == 5.0).all()) and bool((flat[pad + want.numel():] == 5.0).all())


def test_workspace_size_of_long_contexts():
    """The size does not depend on how many blocks a context takes: 10 million tokens in blocks of 1 and of 16."""
    sizes = [pa.pa_prefill_workspace_size(1, 64, 8, 8, 64, bs, 64, 10_000_000, pa.PA_F32) for bs in (1, 16)]
    assert sizes[0] == sizes[1] > 0
