"""Attention weights of cached tokens and eviction by them, from their definitions, in 64 bits.

Tolerances of the weights, derived. Let e = 2^-24 (half a step of fp32). Inputs
are the kernels' own (already rounded); products of 16-bit values are exact in
fp32 and those of fp32 values round once. A score sums D of them in fp32, each
sum off by at most a few e of the magnitudes' total (tensor cores keep at least
fp32's bits for sums of 16 products, with truncation: 2 e a step): under
(2 D + 4) e times A = |scale| sum |q k|, which is what a natural-log score may be
off by; base 2, its scale and the maximum's difference add 4 e of the score's
own size. exp2 is good to 2 units (4 e) and flushes below 2^-126. So a row's
weight p is off by at most p times twice (numerator and the sum under it) the
largest score error, + 16 e; the sum over n tokens rounds at most n / 16 + 16
times (partial sums over lanes, tiles and CTAs): + (n / 16 + 32) e. Weights are
then summed over R rows: R e more, each off by half a step at the most."""
import math

import numpy as np
import torch

E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Paged:
    """Sequences of `lens` tokens in shuffled blocks; slots that hold no token are NaN."""

    def __init__(self, lens, hkv, d, bs, dt, seed, spare=5, max_blocks=None, by=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.hkv, self.d, self.bs = list(lens), hkv, d, bs
        need = [-(-n // bs) for n in lens]
        self.blocks = sum(need) + spare
        perm = rng.permutation(self.blocks)
        width = max_blocks or max(1, max(need))
        # entries past a sequence's blocks are far outside the pool
        self.table = np.full((len(lens), width), 1 << 30, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.k = torch.full((self.blocks, bs, hkv, d), float("nan"), dtype=DT[dt], device="cuda")
        self.v = self.k.clone()
        self.seq_k, self.seq_v = [], []
        for b, n in enumerate(lens):
            ks, vs = ((torch.randn(n, hkv, d, generator=g, device="cuda") * by).to(DT[dt]) for _ in range(2))
            t = torch.arange(n, device="cuda")
            blk = torch.from_numpy(self.table[b].astype(np.int64)).cuda()[t // bs] if n else t
            if n:
                self.k[blk, t % bs], self.v[blk, t % bs] = ks, vs
            self.seq_k.append(ks)
            self.seq_v.append(vs)
        self.tables, self.context_lens = i32(self.table), i32(self.lens)
        self.max_ctx = max(1, max(lens))


def row_weights(q, k, scale, sees):
    """One query token's heads [G, D] over k [n, D] (one KV head): (weights [G, n], error of each), 64 bits."""
    n = k.shape[0]
    q, k = q.double(), k.double()
    s = q @ k.T * scale
    size = (q.abs() @ k.abs().T) * abs(scale)
    s[:, sees:] = -math.inf
    top = s.amax(-1, keepdim=True) if n else s
    p = torch.where(s == -math.inf, torch.zeros_like(s), torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    live = size[:, :sees].amax(-1, keepdim=True) if sees > 0 else torch.zeros_like(total)
    rel = 2 * ((2 * q.shape[-1] + 4) * E * live + 4 * E * live) + 16 * E + (n / 16 + 32) * E
    return p, p * rel + 2.0 ** -120


def weights_after(paged, old, queries, scale, decay, hq, window=0):
    """queries[b] [n_b, Hq, D]: (weights [B, Hkv, S] float64, tolerance), old where nothing is written."""
    want, tol = old.double().clone(), torch.zeros_like(old, dtype=torch.float64)
    g = hq // paged.hkv
    for b, q in enumerate(queries):
        n, ctx = q.shape[0], paged.lens[b]
        if n == 0:
            continue
        count = min(n, window) if window else n
        for h in range(paged.hkv):
            k = paged.seq_k[b][:, h]
            acc, err = torch.zeros(ctx, dtype=torch.float64, device="cuda"), torch.zeros(ctx, dtype=torch.float64, device="cuda")
            for i in range(n - count, n):
                p, e = row_weights(q[i, h * g:(h + 1) * g], k, scale, max(0, min(ctx, ctx - n + i + 1)))
                acc += p.sum(0)
                err += e.sum(0)
            faded = old[b, h, :ctx].double() * decay if decay else torch.zeros_like(acc)
            faded[max(0, ctx - n):] = 0
            want[b, h, :ctx] = acc + faded
            tol[b, h, :ctx] = err + (count * g + 8) * E * acc + 4 * E * faded.abs() + 2.0 ** -120
    return want, tol


def check_weights(got, want, tol):
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), float((got - want).abs().masked_fill(~bad, 0).max()))


def kept_by(w, length, keep, sinks, recent):
    """Positions kept of one head: plain Python, from the definition."""
    keep = min(keep, length)
    recent = min(recent, keep)
    sinks = min(sinks, keep - recent)
    own = set(range(sinks)) | set(range(length - recent, length))
    key = lambda t: -math.inf if math.isnan(w[t]) else w[t]  # noqa: E731
    rest = sorted((t for t in range(length) if t not in own), key=lambda t: (-key(t), t))
    return sorted(own | set(rest[:keep - len(own)]))
