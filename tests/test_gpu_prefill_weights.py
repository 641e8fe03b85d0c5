"""pa_prefill_weights against its definition in 64 bits (tests/weights_cases.py derives the tolerances)."""
import math

import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, Paged, check_weights, i32, weights_after

pytestmark = pytest.mark.gpu


def problem(qlens, lens, hq, hkv, d, bs, dt, seed=0, by=1.0):
    paged = Paged(lens, hkv, d, bs, dt, seed, by=by)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn(sum(qlens), hq, d, generator=g, device="cuda") * 1.5).to(DT[dt])
    old = torch.rand(len(lens), hkv, paged.max_ctx + 3, generator=g, device="cuda")
    for b, (n, c) in enumerate(zip(qlens, lens)):   # the queries' own tokens have no weight yet
        if n:
            old[b, :, max(0, c - n):c] = float("nan")
    start = [0]
    for n in qlens:
        start.append(start[-1] + n)
    return paged, q, old, start


def call(paged, q, old, start, scale, decay, window=0, max_q=None, max_ctx=None):
    w = old.clone()
    B = len(start) - 1
    m = max_q or max(1, max(start[i + 1] - start[i] for i in range(B)))
    c = max_ctx or paged.max_ctx
    ws = torch.full((pa.pa_prefill_weights_workspace_size(B, q.shape[0], q.shape[1], paged.hkv, paged.d, paged.bs, m, c, window),),
                    255, dtype=torch.uint8, device="cuda")
    pa.pa_prefill_weights(w, q, paged.k, paged.tables, paged.context_lens, i32(start), m, c, scale, ws, decay=decay,
                          window=window)
    return w


def split(q, start):
    return [q[a:b] for a, b in zip(start, start[1:])]


SHAPES = [  # query lengths, context lengths, hq, hkv, d, block size
    ((1,), (1,), 1, 1, 64, 16), ((25, 47, 12), (25, 47, 12), 4, 4, 64, 16), ((3, 0, 70), (90, 40, 70), 8, 2, 128, 16),
    ((128, 129), (128, 400), 4, 4, 128, 32), ((33,), (1000,), 12, 3, 64, 7), ((5, 64, 1), (700, 65, 300), 16, 2, 128, 1),
    ((20, 20), (20, 515), 40, 2, 64, 24), ((7,), (2100,), 64, 1, 128, 256), ((300,), (300,), 6, 6, 128, 8),
    ((2, 17, 40), (5, 18, 1200), 8, 8, 64, 64), ((65,), (257,), 9, 1, 64, 4),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("decay,window", [(1.0, 0), (0.0, 16), (0.5, 1), (0.0, 0)])
def test_matches_the_definition(shape, dt, decay, window):
    qlens, lens, hq, hkv, d, bs = shape
    paged, q, old, start = problem(qlens, lens, hq, hkv, d, bs, dt)
    if decay == 0.0:   # not read (but kept where no query token is)
        for b, (n, c) in enumerate(zip(qlens, lens)):
            if n:
                old[b, :, :c] = float("nan")
    scale = d ** -0.5
    w = call(paged, q, old, start, scale, decay, window)
    check_weights(w, *weights_after(paged, old, split(q, start), scale, decay, hq, window))


def test_one_query_token_is_the_decode_step():
    lens = (800, 33, 1)
    paged, q, old, start = problem((1, 1, 1), lens, 8, 2, 128, 16, "bf16", 3)
    w = call(paged, q, old, start, 0.1, 1.0)
    out, got = torch.empty_like(q), old.clone()
    ws = torch.empty(pa.pa_decode_weights_workspace_size(3, 8, 2, 128, 16, 800), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, got, q, paged.k, paged.v, paged.tables, paged.context_lens, 800, 0.1, ws)
    assert torch.allclose(w, got, rtol=2e-5, atol=1e-9, equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_peaked_rows_and_infinite_scores(dt):
    paged, q, old, start = problem((40, 40, 40), (200, 200, 200), 8, 2, 64, 16, dt, 5)
    old = torch.zeros_like(old)
    t, bs = paged.table, paged.bs
    q[40:].abs_().add_(0.1)
    paged.k[int(t[0, 3]), 5] *= 100
    paged.seq_k[0][3 * bs + 5] *= 100
    paged.k[int(t[1, 1]), 1, 0] = -math.inf      # its score is -inf: it weighs nothing
    paged.k[int(t[2, 2]), 0, 0] = math.nan       # every row sees it: its head's weights are NaN
    w = call(paged, q, old, start, 0.125, 1.0)
    want, tol = weights_after(paged, old, split(q, start), 0.125, 1.0, 8)
    check_weights(w[0], want[0], tol[0])
    assert bool((w[1, 0, 17] == 0).all()) and bool(w[1].isfinite().all())
    assert bool(w[2, 0, :200].isnan().all()) and bool(w[2, 1].isfinite().all())


@pytest.mark.parametrize("dt", list(DT))
def test_leading_rows_that_see_nothing(dt):
    """More query tokens than context (the cache was cut): the first ones see nothing and weigh nothing."""
    paged, q, old, start = problem((30,), (12,), 8, 2, 64, 16, dt, 6)
    old = torch.full_like(old, float("nan"))
    w = call(paged, q, old, start, 0.125, 1.0)
    check_weights(w, *weights_after(paged, old, split(q, start), 0.125, 1.0, 8))


def test_bounds_cut_and_sequences_without_queries_stay():
    paged, q, old, start = problem((10, 0, 10), (300, 40, 90), 8, 2, 64, 16, "bf16", 7)
    old = torch.rand_like(old)
    w = call(paged, q, old, start, 0.125, 0.5, max_ctx=128)     # host bound: what lies past it is not attended
    assert torch.equal(w[0, :, 128:], old[0, :, 128:]) and torch.equal(w[1], old[1])
    assert torch.equal(w[2, :, 90:], old[2, :, 90:])
    added = w[0, :, :128] - 0.5 * old[0, :, :128]
    assert torch.allclose(added.sum(-1), torch.full((2,), 40.0, device="cuda"), rtol=1e-3)
    # a query_start that breaks its contract stays in bounds
    for bad in ([0, 10, -5, 20], [0, 1 << 30, 10, 20], [7, 3, 2, 1], [-4, 0, 0, 50]):
        call(paged, q, old, bad, 0.125, 0.5, max_q=16)
    torch.cuda.synchronize()


def test_long_context_splits_and_many_rows():
    for qlens, lens, hq, hkv, d, dt, window in (((4,), (20011,), 8, 2, 64, "bf16", 0), ((700, 300), (700, 900), 8, 2, 128, "fp16", 0),
                                                ((900,), (3000,), 16, 4, 128, "bf16", 64), ((1,) * 100, tuple(range(1, 101)), 4, 2, 64, "fp16", 0)):
        paged, q, old, start = problem(qlens, lens, hq, hkv, d, 16, dt, 9)
        w = call(paged, q, old, start, d ** -0.5, 1.0, window)
        check_weights(w, *weights_after(paged, old, split(q, start), d ** -0.5, 1.0, hq, window))
        assert torch.equal(w.nan_to_num(7.0), call(paged, q, old, start, d ** -0.5, 1.0, window).nan_to_num(7.0))


@pytest.mark.parametrize("dt", list(DT))
def test_a_block_outside_the_pool_reads_as_zeros(dt):
    paged, q, old, start = problem((30, 9), (200, 9), 8, 2, 128, 16, dt, 12)
    old = torch.zeros_like(old)
    for entry, bad in ((2, paged.blocks + 7), (5, -1), (12, 1 << 29)):   # (200 tokens: the last block is cut)
        paged.tables[0, entry] = bad
        paged.seq_k[0][16 * entry:16 * entry + 16] = 0
    w = call(paged, q, old, start, 0.1, 1.0)
    check_weights(w, *weights_after(paged, old, split(q, start), 0.1, 1.0, 8))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_many_units_of_every_shape(dt):
    """More (sequence, head, tile) units than SMs, contexts of an odd number of tiles among them, so that what a
    CTA looks ahead to differs from unit to unit."""
    lens = [130, 300, 77, 257, 513, 1, 700] * 9
    qlens = [5, 300, 77, 2, 60, 1, 130] * 9
    paged, q, old, start = problem(qlens, lens, 8, 4, 64, 16, dt, 13)
    for window in (0, 3):
        w = call(paged, q, old, start, 0.125, 1.0, window)
        check_weights(w, *weights_after(paged, old, split(q, start), 0.125, 1.0, 8, window))


def test_captured_and_replayed():
    paged, q, old, start = problem((130, 64), (1300, 64), 16, 4, 128, 16, "bf16", 11)
    old = torch.rand_like(old)
    want = call(paged, q, old, start, 0.09, 0.5)
    w, qs = old.clone(), i32(start)
    ws = torch.empty(pa.pa_prefill_weights_workspace_size(2, 194, 16, 4, 128, 16, 130, 1300), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill_weights(w, q, paged.k, paged.tables, paged.context_lens, qs, 130, 1300, 0.09, ws, decay=0.5)
    for _ in range(2):
        w.copy_(old)
        graph.replay()
        assert torch.equal(w, want)
