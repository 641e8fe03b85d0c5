"""pa_decode_weights: its outputs against pa_decode's definition and its weights against theirs, in 64 bits
(tests/weights_cases.py derives the tolerances)."""
import math

import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, E, Paged, check_weights, i32, weights_after

pytestmark = pytest.mark.gpu


def call(paged, q, old, scale, decay, out_dt=torch.float32, max_ctx=None, ws=None):
    B, hq, d = q.shape
    out = torch.full((B, hq, d), float("nan"), dtype=out_dt, device="cuda")
    w = old.clone()
    m = max_ctx or paged.max_ctx
    if ws is None:
        ws = torch.full((pa.pa_decode_weights_workspace_size(B, hq, paged.hkv, d, paged.bs, m),), 255, dtype=torch.uint8,
                        device="cuda")
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, m, scale, ws, decay=decay)
    return out, w


def out64(paged, q, scale):
    B, hq, d = q.shape
    g = hq // paged.hkv
    want, size = (torch.zeros(B, hq, d, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, n in enumerate(paged.lens):
        if n == 0:
            continue
        for h in range(hq):
            k, v = paged.seq_k[b][:, h // g].double(), paged.seq_v[b][:, h // g].double()
            s = q[b, h].double() @ k.T * scale
            rel = 2 * (2 * d + 8) * E * float((q[b, h].double().abs() @ k.abs().T).max() * abs(scale)) + 64 * E + n / 8 * E
            p = torch.softmax(s, -1)
            want[b, h], size[b, h] = p @ v, (p @ v.abs()) * (rel + 2.0 ** -15)   # V's weights: two 16-bit parts
    return want, size


def check_out(out, want, size):
    eps = torch.finfo(out.dtype).eps
    err = (out.double() - want).abs()
    tol = size + eps / 2 * (want.abs() + size) + 2.0 ** -25
    assert bool((err <= tol).all()), float((err - tol).max())


def problem(lens, hq, hkv, d, bs, dt, seed=0, extra=3, **kw):
    paged = Paged(lens, hkv, d, bs, dt, seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn(len(lens), hq, d, generator=g, device="cuda") * 1.5).to(DT[dt])
    old = torch.rand(len(lens), hkv, paged.max_ctx + extra, generator=g, device="cuda")
    for b, n in enumerate(lens):   # the newest token's entry holds nothing yet
        if n:
            old[b, :, n - 1] = float("nan")
    return paged, q, old


SHAPES = [  # lens, hq, hkv, d, block size
    ((1,), 1, 1, 64, 16), ((25, 47, 12), 4, 4, 64, 16), ((0, 5, 0, 33), 8, 2, 128, 16), ((700, 3, 1999), 32, 8, 128, 16),
    ((130,), 6, 6, 64, 1), ((97, 128), 12, 3, 128, 7), ((1000, 15, 16, 17), 8, 8, 64, 32), ((300, 299), 40, 2, 128, 24),
    ((511, 64), 16, 1, 64, 256), ((9000,), 8, 8, 128, 16), ((4100,), 14, 2, 128, 8), ((515, 33), 10, 10, 64, 4),
    ((2500, 2499, 100), 71, 1, 64, 16),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
def test_matches_the_definition(shape, dt, decay):
    lens, hq, hkv, d, bs = shape
    paged, q, old = problem(lens, hq, hkv, d, bs, dt)
    if decay == 0.0:
        old.fill_(float("nan"))   # not read
    scale = d ** -0.5
    out, w = call(paged, q, old, scale, decay, out_dt=DT[dt])
    check_out(out, *out64(paged, q, scale))
    check_weights(w, *weights_after(paged, old, [x[None] if n else x[None][:0] for x, n in zip(q, lens)], scale, decay, hq))


def test_agrees_with_the_decode_and_repeats_bit_for_bit():
    paged, q, old = problem((4164,) * 3 + (77, 1200), 32, 8, 128, 16, "bf16", 3)
    out, w = call(paged, q, old, 0.088, 1.0)
    want = torch.empty_like(out)
    pa.pa_decode(want, q, paged.k, paged.v, paged.tables, paged.context_lens, paged.max_ctx, 0.088)
    assert float((out - want).abs().max()) <= 1e-4
    for _ in range(3):
        again = call(paged, q, old, 0.088, 1.0)
        assert torch.equal(out, again[0]) and torch.equal(w[~w.isnan()], again[1][~again[1].isnan()])
    # a row's weights add up to one: over the group's heads, decay 0
    _, w = call(paged, q, torch.zeros_like(old), 0.088, 0.0)
    assert torch.allclose(w.sum(-1), torch.full_like(w.sum(-1), 4.0), rtol=1e-4)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_peaked_rows_infinite_and_nan_scores(dt):
    paged, q, old = problem((200, 200, 200, 64), 8, 2, 64, 16, dt, 5)
    old = torch.zeros_like(old)
    bs, t = paged.bs, paged.table
    # sequence 0: one key a hundred times the others; 1: one key of -inf (and q of one sign: its score is -inf);
    # 2: a NaN key; all of sequence 3's scores -inf: its rows are zeros and weigh nothing
    q[1:].abs_().add_(0.1)
    for s, tok, val in ((1, 17, -math.inf), (2, 100, math.nan)):
        paged.k[int(t[s, tok // bs]), tok % bs, 0] = val
    paged.k[int(t[0, 3]), 5] *= 100
    paged.seq_k[0][3 * bs + 5] *= 100
    for tok in range(64):
        paged.k[int(t[3, tok // bs]), tok % bs] = -math.inf
    out, w = call(paged, q, old, 0.125, 1.0)
    want, tol = weights_after(paged, old, [x[None] for x in q], 0.125, 1.0, 8)
    check_weights(w[0], want[0], tol[0])
    assert bool((w[1, 0, 17] == 0).all()) and bool(w[1].isfinite().all())
    assert bool(w[2, 0, :200].isnan().all()) and bool(w[2, 1].isfinite().all())
    assert bool((w[3, :, :64] == 0).all()) and bool((out[3] == 0).all())


def test_bounds_cut_and_rows_past_the_context_stay():
    paged, q, old = problem((300, 40), 8, 2, 64, 16, "bf16", 7)
    old = torch.rand_like(old)
    out, w = call(paged, q, old, 0.125, 1.0, max_ctx=128)       # host bound: what lies past it is not attended
    assert torch.equal(w[0, :, 128:], old[0, :, 128:]) and torch.equal(w[1, :, 40:], old[1, :, 40:])
    assert torch.allclose((w - old)[0].sum(-1), torch.full((2,), 4.0, device="cuda"), rtol=1e-3)
    paged.context_lens.fill_(-3)
    out, w = call(paged, q, old, 0.125, 1.0)
    assert bool((out == 0).all()) and torch.equal(w, old)
    # a block outside the pool reads as zeros, in keys and values
    paged.context_lens.copy_(i32([300, 40]))
    paged.tables[0, 2] = paged.blocks + 7
    paged.seq_k[0][32:48] = 0
    paged.seq_v[0][32:48] = 0
    old = torch.zeros_like(old)
    out, w = call(paged, q, old, 0.125, 1.0)
    check_weights(w, *weights_after(paged, old, [x[None] for x in q], 0.125, 1.0, 8))
    check_out(out, *out64(paged, q, 0.125))


def test_long_context_few_sequences_and_many_short_ones():
    for lens, hq, hkv, d, dt in (((33000,), 8, 2, 64, "bf16"), ((20011, 9), 4, 1, 128, "fp16"), (tuple(range(1, 180)), 8, 4, 64, "fp16")):
        paged, q, old = problem(lens, hq, hkv, d, 16, dt, 9)
        out, w = call(paged, q, old, d ** -0.5, 1.0)
        check_weights(w, *weights_after(paged, old, [x[None] for x in q], d ** -0.5, 1.0, hq))
        check_out(out, *out64(paged, q, d ** -0.5))


def test_captured_replayed_and_on_a_side_stream():
    paged, q, old = problem((1300, 64, 999), 16, 4, 128, 16, "bf16", 11)
    old = torch.rand_like(old)
    want_out, want_w = call(paged, q, old, 0.09, 0.5)
    out, w = torch.empty_like(want_out), old.clone()
    ws = torch.empty(pa.pa_decode_weights_workspace_size(3, 16, 4, 128, 16, paged.max_ctx), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, paged.max_ctx, 0.09, ws, decay=0.5)
    for _ in range(2):
        w.copy_(old)
        graph.replay()
        assert torch.equal(out, want_out) and torch.equal(w, want_w)
    side = torch.cuda.Stream()
    w.copy_(old)
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_decode_weights(out, w, q, paged.k, paged.v, paged.tables, paged.context_lens, paged.max_ctx, 0.09, ws, decay=0.5,
                         stream=side)
    side.synchronize()
    assert torch.equal(out, want_out) and torch.equal(w, want_w)
