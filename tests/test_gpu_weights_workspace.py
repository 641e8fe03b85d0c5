"""pa_prefill_weights with a workspace sized for other calls: one that was asked for with larger arguments will do for
smaller ones, whatever the work is cut into at either size, and what does not fit is cut into fewer pieces."""
import itertools

import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from weights_cases import DT, Paged, check_weights, i32, weights_after

pytestmark = pytest.mark.gpu


def size(B, T, hq, hkv, d, bs, q, c, window):
    return pa.pa_prefill_weights_workspace_size(B, T, hq, hkv, d, bs, q, c, window)


def run(paged, q, start, window, bytes_given, decay=0.0):
    B, n = len(start) - 1, max(b - a for a, b in zip(start, start[1:]))
    w = torch.zeros(B, paged.hkv, paged.max_ctx, device="cuda")
    guard = torch.full((bytes_given + 4096,), 171, dtype=torch.uint8, device="cuda")
    pa.pa_prefill_weights(w, q, paged.k, paged.tables, paged.context_lens, i32(start), n, paged.max_ctx, 0.1,
                          guard[:bytes_given], decay=decay, window=window)
    assert bool((guard[bytes_given:] == 171).all())     # nothing is written past it
    return w


def least(B, T, hq, q, window):
    """What the call needs at any size, from the sizes alone: the rows' two numbers, the one, four pieces'."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    rows = min(B * (min(window, q) if window else q), T) * hq
    return 256 + up(8 * rows) + up(4 * rows) + up(32 * rows) + up(4 * 4096)


@pytest.mark.parametrize("window", [0, 32])
def test_a_batch_that_shrinks_keeps_its_buffer(window):
    """The buffer of 16 sequences, for any smaller batch of the same prompts."""
    hq, hkv, d, bs, n = 8, 2, 64, 16, 2100
    given = size(16, 16 * n, hq, hkv, d, bs, n, n, window) if window else size(16, 16 * 200, hq, hkv, d, bs, 200, n, 0)
    qlen = n if window else 200
    for B in (1, 3, 7, 13, 14, 15, 16):
        paged = Paged((n,) * B, hkv, d, bs, "bf16", B)
        g = torch.Generator(device="cuda").manual_seed(B)
        q = torch.randn(B * qlen, hq, d, generator=g, device="cuda").bfloat16()
        start = [i * qlen for i in range(B + 1)]
        got = run(paged, q, start, window, given)
        own = run(paged, q, start, window, size(B, B * qlen, hq, hkv, d, bs, qlen, n, window))
        # both are sums of the same terms in another order: each within (n / 16 + 64 + rows) 2^-24 of the exact one
        rows = (window or qlen) * (hq // hkv)
        assert bool(((got - own).abs() <= 2 * (n / 16 + 64 + rows) * 2.0 ** -24 * own + 2.0 ** -100).all())


def test_the_size_covers_every_smaller_call():
    batches, queries, contexts, heads = (1, 2, 15, 16, 20, 300), (1, 31, 130, 2000), (1, 200, 4100, 40000), ((8, 8), (32, 8), (64, 1))
    for B, q, c, (hq, hkv), window in itertools.product(batches, queries, contexts, heads, (0, 1, 32)):
        if q > c:
            continue
        given = size(B, B * q, hq, hkv, 128, 16, q, c, window)
        assert given >= least(B, B * q, hq, q, window)   # and that grows with every argument


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("qlens,lens,hq,window", [((4,), (20011,), 8, 0), ((700, 300), (700, 900), 8, 0), ((900,), (3000,), 16, 64),
                                                  ((40,), (9000,), 4, 0)])
def test_the_least_that_is_needed_will_do(dt, qlens, lens, hq, window):
    """Pieces of contexts and of rows given up, one after another, down to none."""
    paged = Paged(lens, 2, 64, 16, dt, 31)
    g = torch.Generator(device="cuda").manual_seed(32)
    q = torch.randn(sum(qlens), hq, 64, generator=g, device="cuda").to(DT[dt])
    start = [0]
    for n in qlens:
        start.append(start[-1] + n)
    low = least(len(lens), sum(qlens), hq, max(qlens), window)
    full = size(len(lens), sum(qlens), hq, 2, 64, 16, max(qlens), max(lens), window)
    want, tol = weights_after(paged, torch.zeros(len(lens), 2, max(lens), device="cuda"),
                              [q[a:b] for a, b in zip(start, start[1:])], 0.1, 0.0, hq, window)
    for given in sorted({low, (low + full) // 2, (3 * low + full) // 4, max(low, full - 1), full}):
        check_weights(run(paged, q, start, window, given), want, tol)
    with pytest.raises(pa.PAError) as e:   # the two numbers of each row alone do not fit
        run(paged, q, start, window, 256 + 8 * min(sum(qlens), len(lens) * (window or max(qlens))) * hq - 16)
    assert e.value.status == pa.PA_ERR_WORKSPACE
