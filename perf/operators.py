"""What the rotary-position and prefill operators are measured on.

Four operators of the paged cache's prompt and step path:

  rope             pa_rope: heads rotated by their token's position
  rope_and_cache   pa_rope_and_cache: queries and keys rotated, keys and values
                   written into their slots of the paged cache
  prefill          pa_prefill: several query tokens a sequence against the paged
                   cache, causal (prompts, chunks of prompts, verified drafts)
  cross            pa_cross_attention: query tokens against an encoder's states of
                   another length

``own`` False computes them with elementary torch operations in 32 bits (angles
in 64), True calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
WORKSPACE_BYTES = 64 << 20   # more than pa_prefill_workspace_size() asks for at any size here


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # The rotation alone, on the query and key heads of a fused projection's output
        # (32 + 8 heads beside 8 value heads): a prompt chunk of 8,192 tokens.
        dict(name="rope chunk bf16", op="rope", dtype="bf16", tokens=8192, heads=40, pad_heads=8, dim=128, rot=128,
             interleaved=False, transpose=False, base=1e6, scaling="none", scale_by=1.0, last=40960),
        # The gradient of the rotation (its transpose), 32-bit, interleaved pairs, odd token count.
        dict(name="rope transposed fp32", op="rope", dtype="fp32", tokens=2047, heads=16, pad_heads=0, dim=64, rot=64,
             interleaved=True, transpose=True, base=1e4, scaling="none", scale_by=1.0, last=2047),
        # One decode step of the 16-sequence Qwen3-8B layer: 16 tokens, latency counts.
        dict(name="append step bf16", op="rope_and_cache", dtype="bf16", tokens=16, heads=32, kv_heads=8, dim=128,
             rot=128, block=16, padding=0, interleaved=False, base=1e6, scaling="none", scale_by=1.0, last=4164),
        # Four prompts of 4,100 tokens of that layer, written into the cache.
        dict(name="append prompts bf16", op="rope_and_cache", dtype="bf16", tokens=16400, heads=32, kv_heads=8, dim=128,
             rot=128, block=16, padding=0, interleaved=False, base=1e6, scaling="none", scale_by=1.0, last=4100),
        # A padded batch with half of each head rotated, interleaved, positions past the trained
        # length (frequencies blended by parts): the tail of the batch is padding.
        dict(name="append padded fp16", op="rope_and_cache", dtype="fp16", tokens=5000, heads=32, kv_heads=8, dim=128,
             rot=64, block=32, padding=333, interleaved=True, base=1e4, scaling="yarn", scale_by=16.0, last=65536),
        # The 25 / 47 / 12-token toy's prompts, 32-bit: the smallest call.
        dict(name="prefill toy fp32", op="prefill", dtype="fp32", seqs=3, lens="25,47,12", q_lo=0, q_hi=0, past_lo=0,
             past_hi=0, heads=4, kv_heads=4, dim=64, block=16, lens_seed=0),
        # Four drafted tokens a sequence verified over the Qwen3-8B layer's 4,164-token contexts:
        # reads the cache once, a decode step's cost.
        dict(name="verify drafts bf16", op="prefill", dtype="bf16", seqs=16, lens="", q_lo=4, q_hi=4, past_lo=4160,
             past_hi=4160, heads=32, kv_heads=8, dim=128, block=16, lens_seed=0),
        # Four whole prompts of 4,100 tokens: causal, bound by the matrix products.
        dict(name="prefill prompts bf16", op="prefill", dtype="bf16", seqs=4, lens="", q_lo=4100, q_hi=4100, past_lo=0,
             past_hi=0, heads=32, kv_heads=8, dim=128, block=16, lens_seed=0),
        # Continuous batching: 64 sequences, chunks of 1 to 512 tokens behind pasts of up to 3,584.
        dict(name="prefill ragged fp16", op="prefill", dtype="fp16", seqs=64, lens="", q_lo=1, q_hi=512, past_lo=0,
             past_hi=3584, heads=32, kv_heads=8, dim=128, block=32, lens_seed=5),
        # The last 2,048-token chunk of a 32,768-token prompt, 64 query heads.
        dict(name="prefill long bf16", op="prefill", dtype="bf16", seqs=1, lens="", q_lo=2048, q_hi=2048,
             past_lo=30720, past_hi=30720, heads=64, kv_heads=8, dim=128, block=16, lens_seed=0),
        # A decoder's whole target against an encoder's 1,500 states, one head per head.
        dict(name="cross target bf16", op="cross", dtype="bf16", seqs=8, q_lo=300, q_hi=448, ctx_lo=1500, ctx_hi=1500,
             heads=16, kv_heads=16, dim=64, lens_seed=7),
        # One decoder token a sequence against encoder states of ragged lengths.
        dict(name="cross step fp16", op="cross", dtype="fp16", seqs=64, q_lo=1, q_hi=1, ctx_lo=200, ctx_hi=1500,
             heads=16, kv_heads=16, dim=64, lens_seed=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_and_cache", "prefill", "prefill", "cross", "cross"])
    dim = rng.choice([64, 128])
    pos = dict(interleaved=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]), scaling=rng.choice(["none", "linear", "yarn"]),
               scale_by=rng.choice([2.0, 8.0, 32.0]), rot=rng.choice([dim, dim // 2, dim // 4]))
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "rope":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=tokens, heads=rng.randint(1, 40),
                    pad_heads=rng.choice([0, 3, 8]), dim=dim, transpose=rng.random() < 0.4,
                    last=_log(rng, tokens + 1, 131072), **pos)
    if op == "rope_and_cache":
        tokens = _log(rng, 1, 16000)
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=tokens, heads=kv_heads * rng.choice([1, 2, 4]),
                    kv_heads=kv_heads, dim=dim, block=rng.choice([8, 16, 32, 64]), padding=rng.choice([0, tokens // 7]),
                    last=_log(rng, tokens + 1, 131072), **pos)
    dtype = rng.choice(["bf16", "fp16"])
    heads = kv_heads * rng.choice([1, 2, 4, 6, 8])
    seed = rng.randint(0, 1 << 20)
    if op == "prefill":
        q_hi = _log(rng, 1, 4096)
        past_hi = _log(rng, 16, 30000)
        seqs = _log(rng, 1, 64)
        # scores of the padded batch: at most those of the largest listed case
        while seqs > 1 and seqs * heads * q_hi * (q_hi + past_hi) > 3e9:
            seqs -= 1
        while heads * q_hi * (q_hi + past_hi) > 3e9:
            past_hi //= 2
            q_hi = q_hi * 3 // 4
        return dict(op=op, dtype=dtype, seqs=seqs, lens="", q_lo=max(1, q_hi // rng.choice([1, 4])), q_hi=q_hi,
                    past_lo=past_hi // rng.choice([1, 4]), past_hi=past_hi, heads=heads, kv_heads=kv_heads, dim=dim,
                    block=rng.choice([8, 16, 32, 64, 128]), lens_seed=seed)
    q_hi = _log(rng, 1, 512)
    ctx_hi = _log(rng, 16, 3000)
    return dict(op=op, dtype=dtype, seqs=_log(rng, 1, 64), q_lo=max(1, q_hi // 2), q_hi=q_hi, ctx_lo=max(1, ctx_hi // 3),
                ctx_hi=ctx_hi, heads=heads, kv_heads=kv_heads, dim=dim, lens_seed=seed)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _lens(case):
    """(query lengths, context lengths) of an attention case."""
    rng = np.random.default_rng(case["lens_seed"])
    if case["op"] == "cross":
        q = rng.integers(case["q_lo"], case["q_hi"] + 1, case["seqs"])
        return q, rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["seqs"])
    if case["lens"]:
        q = np.array([int(x) for x in case["lens"].split(",")])
        return q, q.copy()
    q = rng.integers(case["q_lo"], case["q_hi"] + 1, case["seqs"])
    return q, q + rng.integers(case["past_lo"], case["past_hi"] + 1, case["seqs"])


def _frequencies(case):
    """(radians a position for each pair, factor on cos and sin), in 64 bits."""
    r, base, s = case["rot"], case["base"], case["scale_by"]
    f = base ** (-2.0 * np.arange(r // 2, dtype=np.float64) / r)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "yarn":   # fast pairs kept, slow ones interpolated, a ramp between (trained length 4,096)
        edge = [r * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
        ramp = np.clip((np.arange(r // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    return f, 1.0


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case, seed=seed)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    d, op = case["dim"], case["op"]
    if op in ("rope", "rope_and_cache"):
        t = case["tokens"]
        freq, s["factor"] = _frequencies(case)
        s["inv_freq"] = torch.from_numpy(freq).cuda()
        pos = rng.integers(0, case["last"], t)
        if op == "rope":
            s["positions"] = i32(pos)
            # the heads to rotate are the first ones of a wider row (a fused projection's output)
            s["x"] = _normal(gen, (t, case["heads"] + case["pad_heads"], d), dt)[:, :case["heads"]]
            s["out"] = torch.zeros(t, case["heads"], d, dtype=dt, device="cuda")
            return s
        live = t - case["padding"]
        pos[live:] = -1
        hq, hkv, bs = case["heads"], case["kv_heads"], case["block"]
        qkv = _normal(gen, (t, hq + 2 * hkv, d), dt)
        s["query"], s["key"], s["value"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        blocks = -(-live // bs) + 8
        table = rng.permutation(blocks)
        slots = np.full(t, -1, np.int64)
        i = np.arange(live)
        slots[:live] = table[i // bs] * bs + i % bs
        s["positions"], s["slots"] = i32(pos), torch.from_numpy(slots).cuda()
        s["k_cache"], s["v_cache"] = (_normal(gen, (blocks, bs, hkv, d), dt) for _ in range(2))
        s["query_out"] = torch.zeros(t, hq, d, dtype=dt, device="cuda")
        return s
    q, ctx = _lens(case)
    hq, hkv, n = case["heads"], case["kv_heads"], case["seqs"]
    t = int(q.sum())
    s["query"] = _normal(gen, (t, hq, d), dt)
    s["query_start"] = i32(np.concatenate([[0], np.cumsum(q)]))
    s["context_lens"] = i32(ctx)
    s["max_q"], s["max_ctx"], s["scale"] = int(q.max()), int(ctx.max()), d ** -0.5
    s["out"] = torch.zeros(t, hq, d, dtype=dt, device="cuda")
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    if op == "cross":
        s["k"], s["v"] = (_normal(gen, (n, s["max_ctx"], hkv, d), dt) for _ in range(2))
        return s
    bs = case["block"]
    need = -(-ctx // bs)
    perm = rng.permutation(int(need.sum()) + 8)
    tables = np.zeros((n, int(need.max())), np.int32)
    at = 0
    for b in range(n):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    s["block_tables"] = i32(tables)
    s["k_cache"], s["v_cache"] = (_normal(gen, (perm.size, bs, hkv, d), dt) for _ in range(2))
    return s


# --------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits
# --------------------------------------------------------------------------
def _rotated(x, positions, inv_freq, factor, rot, interleaved, transpose):
    angle = positions.double()[:, None] * inv_freq[None]
    cos = (angle.cos() * factor).float()[:, None]
    sin = (angle.sin() * factor).float()[:, None]
    if transpose:
        sin = -sin
    y = x.float()
    r = y[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _attended(query, k, v, context_lens, query_start, max_q, scale, causal):
    """query [T, Hq, D] ragged; k, v [B, L, Hkv, D] padded."""
    t, hq, d = query.shape
    n, length, hkv, _ = k.shape
    g = hq // hkv
    start, q_len = query_start[:-1].long(), query_start.diff().long()
    i = torch.arange(max_q, device=query.device)
    rows = (start[:, None] + i).clamp(max=t - 1)
    q = query[rows].float().view(n, max_q, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, max_q * g, d)
    j = torch.arange(length, device=query.device)
    ctx = context_lens.long()[:, None]
    dead = (j >= ctx)[:, :, None, None]
    kf = k.float().permute(0, 2, 3, 1)
    vf = v.float().masked_fill(dead, 0.0).permute(0, 2, 1, 3)
    sees = (ctx - q_len[:, None] + i + 1) if causal else ctx.expand(n, max_q)
    sees = torch.minimum(sees, ctx)
    scores = torch.matmul(q, kf).mul_(scale).view(n, hkv, max_q, g, length)
    scores.masked_fill_((j >= sees[:, :, None])[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_().view(n, hkv, max_q * g, length)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, vf) / total.clamp(min=1e-38)
    o = o.view(n, hkv, max_q, g, d).permute(0, 2, 1, 3, 4).reshape(n, max_q, hq, d)
    token = torch.arange(t, device=query.device)
    seq = torch.searchsorted(query_start[1:].long(), token, right=True)
    return o[seq, token - start[seq]].to(query.dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import paged_kv_cache_121_gb300 as pa
        layout = pa.PA_ROPE_INTERLEAVED if c.get("interleaved") else pa.PA_ROPE_HALF
        if op == "rope":
            pa.pa_rope(s["out"], s["x"], s["positions"], s["inv_freq"], layout=layout, factor=s["factor"],
                       transpose=c["transpose"])
            return s["out"]
        if op == "rope_and_cache":
            pa.pa_rope_and_cache(s["query_out"], s["query"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"],
                                 s["positions"], s["inv_freq"], layout=layout, factor=s["factor"])
            return s["query_out"], s["k_cache"], s["v_cache"]
        if op == "prefill":
            pa.pa_prefill(s["out"], s["query"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                          s["query_start"], s["max_q"], s["max_ctx"], s["scale"], causal=True, workspace=s["workspace"])
            return s["out"]
        pa.pa_cross_attention(s["out"], s["query"], s["k"], s["v"], s["context_lens"], s["query_start"], s["max_q"],
                              s["max_ctx"], s["scale"], workspace=s["workspace"])
        return s["out"]
    if op == "rope":
        s["out"].copy_(_rotated(s["x"], s["positions"], s["inv_freq"], s["factor"], c["rot"], c["interleaved"], c["transpose"]))
        return s["out"]
    if op == "rope_and_cache":
        args = (s["positions"], s["inv_freq"], s["factor"], c["rot"], c["interleaved"], False)
        padding = (s["positions"] < 0)[:, None, None]
        s["query_out"].copy_(torch.where(padding, s["query_out"], _rotated(s["query"], *args)))
        hkv, d = c["kv_heads"], c["dim"]
        k, v = s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)
        # padding tokens are the last ones: the tokens before them have distinct slots
        live = c["tokens"] - c["padding"]
        slots = s["slots"][:live]
        k[slots] = _rotated(s["key"], *args)[:live]
        v[slots] = s["value"][:live]
        return s["query_out"], s["k_cache"], s["v_cache"]
    if op == "prefill":
        n, hkv, d = c["seqs"], c["kv_heads"], c["dim"]
        table = s["block_tables"].long()
        k = s["k_cache"][table].view(n, -1, hkv, d)[:, :s["max_ctx"]]
        v = s["v_cache"][table].view(n, -1, hkv, d)[:, :s["max_ctx"]]
        return _attended(s["query"], k, v, s["context_lens"], s["query_start"], s["max_q"], s["scale"], True)
    return _attended(s["query"], s["k"], s["v"], s["context_lens"], s["query_start"], s["max_q"], s["scale"], False)


# --------------------------------------------------------------------------
# work, and the definition in 64 bits
# --------------------------------------------------------------------------
def work(case):
    e, d, op = BYTES[case["dtype"]], case["dim"], case["op"]
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        return dict(bytes=2 * t * h * d * e + 4 * t + 4 * case["rot"], flops=3 * t * h * case["rot"])
    if op == "rope_and_cache":
        t, hq, hkv = case["tokens"] - case["padding"], case["heads"], case["kv_heads"]
        return dict(bytes=2 * t * (hq + 2 * hkv) * d * e + 12 * case["tokens"] + 4 * case["rot"],
                    flops=3 * t * (hq + hkv) * case["rot"])
    q, ctx = _lens(case)
    hq, hkv = case["heads"], case["kv_heads"]
    if op == "prefill":   # token i of a query sees ctx - q + i + 1 tokens
        pairs = int((q * (ctx - q) + q * (q + 1) // 2).sum())
        table = 4 * int((-(-ctx // case["block"])).sum())
    else:
        pairs, table = int((q * ctx).sum()), 0
    return dict(bytes=2 * int(q.sum()) * hq * d * e + 2 * int(ctx.sum()) * hkv * d * e + table + 8 * case["seqs"],
                flops=4 * d * hq * pairs)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["dim"]
    if op in ("rope", "rope_and_cache"):
        half = case["rot"] // 2
        theta = torch.outer(s["positions"].double(), s["inv_freq"])
        # a pair is a complex number, turned by e^(i theta) (its conjugate for the transpose)
        turn = torch.polar(torch.full_like(theta, s["factor"]), -theta if case.get("transpose") else theta)

        def turned(x):
            y = x.double().clone()
            first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
            second = first + (1 if case["interleaved"] else half)
            z = torch.complex(y[:, :, first], y[:, :, second]) * turn[:, None]
            y[:, :, first], y[:, :, second] = z.real, z.imag
            return y

        if op == "rope":
            return turned(s["x"])
        live = case["tokens"] - case["padding"]
        q = s["query_out"].double()
        q[:live] = turned(s["query"])[:live]
        k, v = s["k_cache"].double(), s["v_cache"].double()
        block, offset = s["slots"][:live] // case["block"], s["slots"][:live] % case["block"]
        k[block, offset] = turned(s["key"])[:live]
        v[block, offset] = s["value"][:live].double()
        return q, k, v
    q_lens, ctx = _lens(case)
    hq, hkv = case["heads"], case["kv_heads"]
    out = torch.zeros(int(q_lens.sum()), hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["seqs"]):
        n, length = int(q_lens[b]), int(ctx[b])
        if op == "prefill":
            where = torch.arange(length, device="cuda")
            blocks = s["block_tables"][b].long()[where // case["block"]]
            k, v = (s[c][blocks, where % case["block"]].double() for c in ("k_cache", "v_cache"))
        else:
            k, v = s["k"][b, :length].double(), s["v"][b, :length].double()
        hidden = None
        if op == "prefill":
            hidden = torch.ones(n, length, dtype=torch.bool, device="cuda").triu(length - n + 1)
        for h in range(hq):
            g = h // (hq // hkv)
            logits = s["query"][at:at + n, h].double() @ k[:, g].T * s["scale"]
            if hidden is not None:
                logits = logits.masked_fill(hidden, -math.inf)
            out[at:at + n, h] = torch.softmax(logits, -1) @ v[:, g]
        at += n
    return out
