"""Scores of any finite size. Queries and keys are constant rows of powers of two
times small whole numbers, so every score is exact in fp32 and differs from the
next kind by far more than the softmax can bridge: a row's output is the plain
average of the values of its highest-scoring tokens.

Tolerance, with A the average of |v| over those tokens: the equal weights rounded
once, numerator alone: u A with u = eps / 2 of a 16-bit cache (fp32: none); the sums
over n tokens in fp32: 2 (n + 16) 2^-23 A; the output rounded: eps / 2 |y|."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from prefill_cases import Case

pytestmark = pytest.mark.gpu

SHAPES = [   # query lengths, context lengths, Hq, Hkv, D, block size
    ([3, 1], [700, 460], 16, 4, 64, 16),            # few rows
    ([20, 5], [1000, 450], 4, 2, 128, 16),          # one row tile
    ([150], [800], 8, 2, 128, 64),                  # two row tiles
    ([100] * 4, [6200, 6100, 17, 6200], 8, 8, 64, 0),   # contexts cut into pieces
]


def check(shape, dt, a, b, sign, spread):
    q, ctx, hq, hkv, d, bs = shape
    c = Case(q, ctx, hq, hkv, d, bs, dt, seed=7, scale=2.0 ** -3 * sign)
    c.query.fill_(a)
    for i, n in enumerate(c.ctx_lens):   # keys b, 2 b or 3 b (or all alike), runs of 150 tokens
        level = 1 + (torch.arange(n, device="cuda") // 150) % 3 if spread else torch.ones(n, device="cuda")
        c.k[i] = (b * level.to(torch.float64)).to(c.dt)[:, None, None].expand(n, hkv, d)
        if bs:
            flat = torch.full((-(-n // bs) * bs, hkv, d), float("nan"), dtype=c.dt, device="cuda")
            flat[:n] = c.k[i]
            c.kc[c.tables_d[i, :-(-n // bs)].long()] = flat.view(-1, bs, hkv, d)
        else:
            c.kc[i, :n] = c.k[i]
    causal = bool(bs)
    u = 0.0 if c.dt == torch.float32 else torch.finfo(c.dt).eps / 2
    for ws in (None, c.workspace()):
        out = c.run(causal, ws).double()
        for i, n in enumerate(c.ctx_lens):
            for t in (0, c.q_lens[i] // 2, c.q_lens[i] - 1):
                sees = n - c.q_lens[i] + t + 1 if causal else n
                if sees <= 0:
                    continue
                keys = c.k[i][:sees, 0, 0].double() * sign
                v = c.v[i][:sees][keys == keys.max()].double().repeat_interleave(hq // hkv, 1)
                want, avg = v.mean(0), v.abs().mean(0)
                tol = (u + 2 * (sees + 16) * 2.0 ** -23) * avg
                tol = tol + torch.finfo(c.dt).eps / 2 * (want.abs() + tol) + 2.0 ** -25
                err = (out[int(c.start[i]) + t] - want).abs()
                assert bool((err <= tol).all()), (i, t, float((err / tol).max()))
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("log2", [20, 22, 23, 28, 33, 64, 100, 118])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_bf16_and_fp32(shape, log2, sign, spread):
    """Scores of about 2^log2 (times head_dim / 8), of one sign or the other."""
    for dt in ("bf16", "fp32"):
        check(SHAPES[shape], dt, 2.0 ** (log2 // 2), 2.0 ** (log2 - log2 // 2), sign, spread)


@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("log2", [20, 22, 23, 26, 29])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_fp16(shape, log2, sign, spread):
    check(SHAPES[shape], "fp16", 2.0 ** 15, 2.0 ** (log2 - 15), sign, spread)
