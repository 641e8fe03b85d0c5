"""Inputs, a 64-bit reference and derived tolerances for pa_prefill and
pa_cross_attention.

Tolerance of one output element, with A = sum_j p_j |v_j| / l (the softmax
average of |v|) and s_max the largest sum |q| |k| of its row:
  * the weights p rounded once to the caches' 16-bit type: u A with u = eps / 2
    (fp32 caches: no such rounding); an fp16 weight below 2^-14 is off by up to
    2^-25 whole instead, where the largest weight is at least 1: 2^-25 sum |v|;
  * a score summed over head_dim products in fp32, in any order: off by at most
    (D + 2) 2^-23 |scale| s_max (2^-23: the tensor cores may truncate), which
    moves every weight by as much relatively, numerator and denominator: twice;
  * the weighted sum and the sum of weights over n tokens in fp32: 2 (n + 16)
    2^-23 A (16: exponentials, rescales, merges);
  * the output rounded to its type: eps / 2 |y| (2^-25 below fp16's normals).
"""
import numpy as np
import torch

import paged_kv_cache_121_gb300 as pa

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


class Case:
    """Ragged queries over a paged (block_size > 0) or contiguous (0) cache; what no sequence owns is NaN."""

    def __init__(self, q_lens, ctx_lens, hq, hkv, d, bs, dt, seed=0, lead=0, trail=0, spare=5, max_states=None,
                 scale=None):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_lens, self.ctx_lens = list(q_lens), list(ctx_lens)
        self.hq, self.hkv, self.d, self.bs, self.dt = hq, hkv, d, bs, DT[dt]
        self.n, self.tokens = len(q_lens), lead + sum(q_lens) + trail
        self.start = np.concatenate([[lead], lead + np.cumsum(q_lens)]).astype(np.int32)
        self.scale = d ** -0.5 if scale is None else scale
        normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(self.dt)  # noqa: E731
        self.query = normal(self.tokens, hq, d)
        self.k = [normal(c, hkv, d) for c in ctx_lens]
        self.v = [normal(c, hkv, d) for c in ctx_lens]
        nan = float("nan")
        if bs:
            need = [-(-c // bs) for c in ctx_lens]
            nb = sum(need) + spare
            perm = rng.permutation(nb).astype(np.int32)
            width = max(need + [1])
            self.tables = rng.choice(np.array([-7, 10 ** 6, nb], np.int32), (self.n, width)).astype(np.int32)
            self.kc = torch.full((nb, bs, hkv, d), nan, dtype=self.dt, device="cuda")
            self.vc = torch.full_like(self.kc, nan)
            at = 0
            for b, c in enumerate(ctx_lens):
                ids = perm[at:at + need[b]]
                at += need[b]
                self.tables[b, :need[b]] = ids
                for cache, rows in ((self.kc, self.k[b]), (self.vc, self.v[b])):
                    if c:
                        flat = torch.full((need[b] * bs, hkv, d), nan, dtype=self.dt, device="cuda")
                        flat[:c] = rows
                        cache[torch.from_numpy(ids).long().cuda()] = flat.view(-1, bs, hkv, d)
            self.tables_d = torch.from_numpy(self.tables).cuda()
        else:
            states = max_states or max(ctx_lens + [1])
            self.kc = torch.full((self.n, states, hkv, d), nan, dtype=self.dt, device="cuda")
            self.vc = torch.full_like(self.kc, nan)
            for b, c in enumerate(ctx_lens):
                self.kc[b, :c], self.vc[b, :c] = self.k[b], self.v[b]
        self.start_d = torch.from_numpy(self.start).cuda()
        self.ctx_d = torch.tensor(self.ctx_lens, dtype=torch.int32, device="cuda")
        self.max_q, self.max_ctx = max(self.q_lens), max(self.ctx_lens)

    def workspace(self, fill=0xFF):
        n = pa.pa_prefill_workspace_size(self.n, self.tokens, self.hq, self.hkv, self.d, self.bs or 16, self.max_q,
                                         self.max_ctx, {torch.bfloat16: 1, torch.float16: 2, torch.float32: 0}[self.dt])
        return torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")

    def run(self, causal, workspace=None, out_dtype=None, out=None, stream=None):
        if out is None:
            out = torch.full((self.tokens, self.hq, self.d), 5.0, dtype=out_dtype or self.dt, device="cuda")
        if self.bs:
            pa.pa_prefill(out, self.query, self.kc, self.vc, self.tables_d, self.ctx_d, self.start_d, self.max_q,
                          self.max_ctx, self.scale, causal=causal, workspace=workspace, stream=stream)
        else:
            assert not causal
            pa.pa_cross_attention(out, self.query, self.kc, self.vc, self.ctx_d, self.start_d, self.max_q,
                                  self.max_ctx, self.scale, workspace=workspace, stream=stream)
        return out

    def check(self, out, causal):
        """Every row against the definition in 64 bits; rows no sequence owns untouched."""
        g = self.hq // self.hkv
        odt = out.dtype
        u_out = torch.finfo(odt).eps / 2
        u_p = 0.0 if self.dt == torch.float32 else torch.finfo(self.dt).eps / 2
        tiny = 2.0 ** -25 if odt == torch.float16 else 0.0
        own = torch.zeros(self.tokens, dtype=torch.bool, device="cuda")
        for b in range(self.n):
            n, c, at = self.q_lens[b], self.ctx_lens[b], int(self.start[b])
            if n == 0:
                continue
            own[at:at + n] = True
            got = out[at:at + n].double()
            assert bool(torch.isfinite(got).all()), (b, "not finite")
            if c == 0:
                assert not bool(got.any()), b
                continue
            q = self.query[at:at + n].double().view(n, self.hkv, g, self.d)
            k, v = self.k[b].double(), self.v[b].double()
            s = torch.einsum("nhgd,chd->hgnc", q, k) * self.scale
            size = torch.einsum("nhgd,chd->hgnc", q.abs(), k.abs()).amax(-1)
            i, j = torch.arange(n, device="cuda"), torch.arange(c, device="cuda")
            if causal:
                s.masked_fill_(j[None] > (c - n + i)[:, None], -float("inf"))
            empty = torch.isinf(s).all(-1) & (s[..., 0] < 0)
            p = torch.softmax(s, -1)
            p.masked_fill_(empty[..., None], 0.0)
            want = torch.einsum("hgnc,chd->nhgd", p, v).reshape(n, self.hq, self.d)
            avg = torch.einsum("hgnc,chd->nhgd", p, v.abs()).reshape(n, self.hq, self.d)
            tol = (u_p + 2 * (c + 16) * 2.0 ** -23) * avg
            tol += (2 * (self.d + 2) * 2.0 ** -23 * abs(self.scale) * size).permute(2, 0, 1).reshape(n, self.hq, 1) * avg
            if self.dt == torch.float16:
                tol += 2.0 ** -25 * v.abs().sum(0).repeat_interleave(g, 0)[None]
            tol = tol + u_out * (want.abs() + tol) + tiny
            err = (got - want).abs()
            assert bool((err <= tol).all()), (b, float((err - tol).max()), float((err / tol).max()))
        assert bool((out[~own] == 5.0).all())
