"""What the operators around a bounded cache are measured on.

A cache that holds the heavy hitters of a long context: queries and keys are
normed and rotated on the way in, each attention call adds the weight that it
gave every cached token to a table, and an eviction keeps the tokens that
weighed most.

  norm_rope        pa_norm_rope: heads normed (root mean square, learned scale)
                   and rotated by their token's position
  norm_rope_grad   pa_norm_rope_backward: its gradients
  norm_rope_cache  pa_norm_rope_and_cache: the same for queries and keys, keys and
                   values written into their slots of the paged cache
  decode_weights   pa_decode_weights: one decode step, and the weight that it gave
                   each cached token
  prefill_weights  pa_prefill_weights: the weights that the queries of a prompt (or
                   the last ones of it) gave each cached token
  evict            pa_evict: each head's heaviest tokens, first and last ones kept,
                   moved together into other blocks

``own`` False computes them with elementary torch operations in 32 bits (angles
in 64), True calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
WORKSPACE_BYTES = 128 << 20   # more than the library's ..._workspace_size() ask for at any size here


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # The query heads of a fused projection's output (32 beside 16 key and value heads), a
        # prompt chunk of 8,192 tokens.
        dict(name="norm rope chunk bf16", op="norm_rope", dtype="bf16", tokens=8192, heads=32, pad_heads=16, dim=128,
             rot=128, interleaved=False, base=1e6, last=40960),
        # 32-bit, interleaved pairs, half of each head rotated, odd token count.
        dict(name="norm rope odd fp32", op="norm_rope", dtype="fp32", tokens=2047, heads=16, pad_heads=0, dim=64,
             rot=32, interleaved=True, base=1e4, last=2047),
        # Training: the gradients of the first case, of the heads and of the learned scale.
        dict(name="norm rope grad bf16", op="norm_rope_grad", dtype="bf16", tokens=8192, heads=32, pad_heads=16, dim=128,
             rot=128, interleaved=False, base=1e6, last=40960),
        # A small 32-bit model's key heads.
        dict(name="norm rope grad fp32", op="norm_rope_grad", dtype="fp32", tokens=1023, heads=8, pad_heads=0, dim=64,
             rot=64, interleaved=True, base=1e4, last=1023),
        # One decode step of the 16-sequence Qwen3-8B layer: 16 tokens, latency counts.
        dict(name="norm append step bf16", op="norm_rope_cache", dtype="bf16", tokens=16, heads=32, kv_heads=8, dim=128,
             rot=128, block=16, padding=0, interleaved=False, base=1e6, last=4164),
        # Four prompts of 4,100 tokens of that layer, the last rows of the batch padding.
        dict(name="norm append prompts bf16", op="norm_rope_cache", dtype="bf16", tokens=16500, heads=32, kv_heads=8,
             dim=128, rot=128, block=16, padding=100, interleaved=False, base=1e6, last=4100),
        # The 25 / 47 / 12-token toy, 32-bit: the smallest decode.
        dict(name="decode toy fp32", op="decode_weights", dtype="fp32", seqs=3, lens="25,47,12", ctx_lo=0, ctx_hi=0,
             heads=4, kv_heads=4, dim=64, block=16, decay=1.0, lens_seed=0),
        # The Qwen3-8B layer's decode step: 16 contexts of 4,164 tokens.
        dict(name="decode layer bf16", op="decode_weights", dtype="bf16", seqs=16, lens="", ctx_lo=4164, ctx_hi=4164,
             heads=32, kv_heads=8, dim=128, block=16, decay=1.0, lens_seed=0),
        # The last 32 queries of 16 prompts of 4,100 tokens vote on what stays of each.
        dict(name="window prompts bf16", op="prefill_weights", dtype="bf16", seqs=16, q_lo=4100, q_hi=4100, past_lo=0,
             past_hi=0, window=32, heads=32, kv_heads=8, dim=128, block=16, decay=0.0, lens_seed=0),
        # Every query counts: ragged chunks of up to 1,500 tokens behind up to 2,500, older weights fading.
        dict(name="chunks ragged fp16", op="prefill_weights", dtype="fp16", seqs=8, q_lo=200, q_hi=1500, past_lo=0,
             past_hi=2500, window=0, heads=32, kv_heads=8, dim=128, block=32, decay=0.95, lens_seed=3),
        # That layer's 16 contexts cut to half their tokens.
        dict(name="evict layer bf16", op="evict", dtype="bf16", seqs=16, ctx_lo=4164, ctx_hi=4164, keep=2048, sinks=4,
             recent=256, kv_heads=8, dim=128, block=16, lens_seed=0),
        # One context of 32,768 tokens cut to an eighth.
        dict(name="evict long fp16", op="evict", dtype="fp16", seqs=1, ctx_lo=32768, ctx_hi=32768, keep=4096, sinks=4,
             recent=512, kv_heads=8, dim=128, block=32, lens_seed=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "norm_rope_cache", "decode_weights", "decode_weights",
                     "prefill_weights", "prefill_weights", "evict", "evict"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op.startswith("norm_rope"):
        tokens = _log(rng, 1, 8192)
        c = dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=tokens, dim=dim,
                 rot=rng.choice([dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]),
                 last=_log(rng, tokens + 1, 131072))
        if op == "norm_rope_cache":
            return dict(heads=kv_heads * rng.choice([1, 2, 4]), kv_heads=kv_heads, block=rng.choice([8, 16, 32, 64]),
                        padding=rng.choice([0, tokens // 7]), **c)
        return dict(heads=rng.randint(1, 32), pad_heads=rng.choice([0, 3, 16]), **c)
    seed = rng.randint(0, 1 << 20)
    heads = kv_heads * rng.choice([1, 2, 4, 6, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"])
    block = rng.choice([8, 16, 32, 64])
    seqs = _log(rng, 1, 64)
    row = kv_heads * dim * BYTES[dtype]
    if op == "decode_weights":
        ctx_hi = _log(rng, 16, 32768)
        while seqs > 1 and seqs * ctx_hi * row > 1.3e8:
            seqs -= 1
        return dict(op=op, dtype=dtype, seqs=seqs, lens="", ctx_lo=max(1, ctx_hi // rng.choice([1, 2, 8])), ctx_hi=ctx_hi,
                    heads=heads, kv_heads=kv_heads, dim=dim, block=block, decay=rng.choice([1.0, 0.9]), lens_seed=seed)
    if op == "evict":
        ctx_hi = _log(rng, 16, 32768)
        while seqs > 1 and seqs * ctx_hi * row > 0.9e8:
            seqs -= 1
        keep = max(8, int(ctx_hi * rng.uniform(0.1, 0.7)))
        return dict(op=op, dtype=dtype, seqs=seqs, ctx_lo=max(1, ctx_hi // rng.choice([1, 2, 8])), ctx_hi=ctx_hi, keep=keep,
                    sinks=rng.choice([0, 4]), recent=rng.choice([0, keep // 8, keep // 2]), kv_heads=kv_heads, dim=dim,
                    block=block, lens_seed=seed)
    q_hi = _log(rng, 1, 2048)
    past_hi = _log(rng, 16, 16384)
    window = rng.choice([0, 16, 32, 64])
    wide = min(q_hi, window) if window else q_hi
    if dtype == "fp32" and wide > 64:
        dtype = "bf16"
    # scores and keys of the padded batch: at most those of the largest listed cases
    while seqs > 1 and (seqs * heads * wide * (q_hi + past_hi) > 2.4e8 or seqs * (q_hi + past_hi) * row > 1.3e8):
        seqs -= 1
    while heads * wide * (q_hi + past_hi) > 2.4e8:
        past_hi //= 2
        q_hi = max(1, q_hi * 3 // 4)
        wide = min(q_hi, window) if window else q_hi
    return dict(op=op, dtype=dtype, seqs=seqs, q_lo=max(1, q_hi // rng.choice([1, 4])), q_hi=q_hi,
                past_lo=past_hi // rng.choice([1, 4]), past_hi=past_hi, window=window, heads=heads, kv_heads=kv_heads,
                dim=dim, block=block, decay=rng.choice([0.0, 1.0, 0.9]), lens_seed=seed)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _lens(case):
    """(query lengths, context lengths) of an attention or eviction case."""
    rng = np.random.default_rng(case["lens_seed"])
    if case["op"] == "prefill_weights":
        q = rng.integers(case["q_lo"], case["q_hi"] + 1, case["seqs"])
        return q, q + rng.integers(case["past_lo"], case["past_hi"] + 1, case["seqs"])
    if case.get("lens"):
        ctx = np.array([int(x) for x in case["lens"].split(",")])
    else:
        ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["seqs"])
    return np.ones_like(ctx), ctx


def _normal(gen, shape, dtype, by=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(by).to(dtype)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _tables(rng, lens, block, spare=8, first=0):
    """Block tables of sequences of `lens` tokens in shuffled blocks first .. , and how many blocks they need."""
    need = -(-lens // block)
    perm = first + rng.permutation(int(need.sum()) + spare)
    tables = np.zeros((lens.size, max(1, int(need.max()))), np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(lens.size):
        tables[b, :need[b]] = perm[at[b]:at[b + 1]]
    return tables, perm.size


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case, seed=seed)
    d, op = case["dim"], case["op"]
    if op.startswith("norm_rope"):
        t, s["eps"] = case["tokens"], 1e-6
        r = case["rot"]
        s["inv_freq"] = torch.from_numpy(case["base"] ** (-2.0 * np.arange(r // 2, dtype=np.float64) / r)).cuda()
        pos = rng.integers(0, case["last"], t)
        if op != "norm_rope_cache":
            wide = (t, case["heads"] + case["pad_heads"], d)
            s["positions"] = _i32(pos)
            s["x"] = _normal(gen, wide, dt, 2.0)[:, :case["heads"]]
            s["weight"] = (1.0 + _normal(gen, (d,), torch.float32, 0.2)).to(dt)
            if op == "norm_rope":
                s["out"] = torch.zeros(t, case["heads"], d, dtype=dt, device="cuda")
                return s
            s["grad_out"] = _normal(gen, (t, case["heads"], d), dt)
            # the heads' part of the fused projection's gradient
            s["grad_x"] = torch.zeros(wide, dtype=dt, device="cuda")[:, :case["heads"]]
            s["grad_weight"] = torch.zeros(d, dtype=torch.float32, device="cuda")
            s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
            return s
        live = t - case["padding"]
        pos[live:] = -1
        hq, hkv, bs = case["heads"], case["kv_heads"], case["block"]
        qkv = _normal(gen, (t, hq + 2 * hkv, d), dt, 2.0)
        s["query"], s["key"], s["value"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["query_weight"], s["key_weight"] = ((1.0 + _normal(gen, (d,), torch.float32, 0.2)).to(dt) for _ in range(2))
        blocks = -(-live // bs) + 8
        table = rng.permutation(blocks)
        slots = np.full(t, -1, np.int64)
        i = np.arange(live)
        slots[:live] = table[i // bs] * bs + i % bs
        s["positions"], s["slots"] = _i32(pos), torch.from_numpy(slots).cuda()
        s["k_cache"], s["v_cache"] = (_normal(gen, (blocks, bs, hkv, d), dt) for _ in range(2))
        s["query_out"] = torch.zeros(t, hq, d, dtype=dt, device="cuda")
        return s
    q, ctx = _lens(case)
    hkv, n, bs = case["kv_heads"], case["seqs"], case["block"]
    tables, blocks = _tables(rng, ctx, bs)
    s["block_tables"], s["context_lens"], s["max_ctx"] = _i32(tables), _i32(ctx), int(ctx.max())
    # what earlier steps left: most tokens weigh little, a few much
    w = torch.rand(n, hkv, s["max_ctx"] + 7, generator=gen, device="cuda").pow_(8).mul_(4.0)
    if op == "evict":
        # (many weights are equal: whole steps of 1 / 1,024, and tokens that never weighed anything)
        s["weights"] = torch.where(w < 0.5, (w * 1024).floor() / 1024, w)
        keep = np.minimum(case["keep"], ctx)
        new_tables, total = _tables(rng, keep, bs, first=blocks)
        s["new_tables"], s["keep_lens"] = _i32(new_tables), _i32(np.full(n, case["keep"]))
        s["k_cache"], s["v_cache"] = (_normal(gen, (blocks + total, bs, hkv, d), dt) for _ in range(2))
        s["kept"] = torch.zeros(n, hkv, case["keep"], dtype=torch.int32, device="cuda")
        s["new_weights"] = torch.zeros_like(w)
        return s
    s["weights"] = w
    s["k_cache"], s["v_cache"] = (_normal(gen, (blocks, bs, hkv, d), dt) for _ in range(2))
    hq, t = case["heads"], int(q.sum())
    s["query"] = _normal(gen, (t, hq, d), dt, 1.5)
    s["query_start"] = _i32(np.concatenate([[0], np.cumsum(q)]))
    s["max_q"], s["scale"] = int(q.max()), d ** -0.5
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    if op == "decode_weights":
        s["out"] = torch.zeros(n, hq, d, dtype=dt, device="cuda")
    return s


# --------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits
# --------------------------------------------------------------------------
def _turn(s, c, transpose=False):
    angle = s["positions"].double()[:, None] * s["inv_freq"][None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return cos, -sin if transpose else sin


def _rotated(y, turn, rot, interleaved):
    cos, sin = turn
    r = y[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1)


def _normed(x, weight, eps):
    y = x.float()
    return y * (y.square().mean(-1, keepdim=True) + eps).rsqrt() * weight.float()


def _norm_rope_grad(s, c):
    x, w = s["x"].float(), s["weight"].float()
    g = _rotated(s["grad_out"].float(), _turn(s, c, True), c["rot"], c["interleaved"])
    inv = (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
    unit = x * inv
    wg = g * w
    grad_x = inv * (wg - unit * (wg * unit).mean(-1, keepdim=True))
    return grad_x, (g * unit).sum((0, 1))


def _attended(s, c, first, count, max_count, with_out):
    """The softmax weights that `count` query rows of each sequence from row `first` on (its context's
    last ones) gave each cached token, summed over the rows and the query heads of each KV head
    [B, Hkv, L]; and the rows' outputs, for a count of one."""
    query, n, hq, hkv, d = s["query"], c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    g, length = hq // hkv, s["max_ctx"]
    table = s["block_tables"].long()
    k = s["k_cache"][table].view(n, -1, hkv, d)[:, :length].float().permute(0, 2, 3, 1)
    i = torch.arange(max_count, device=query.device)
    j = torch.arange(length, device=query.device)
    ctx = s["context_lens"].long()
    rows = (first[:, None] + i).clamp(max=query.shape[0] - 1)
    q = query[rows].float().view(n, max_count, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, max_count * g, d)
    sees = ctx[:, None] - count[:, None] + i + 1
    scores = torch.matmul(q, k).mul_(s["scale"]).view(n, hkv, max_count, g, length)
    scores.masked_fill_((j >= sees[:, :, None])[:, None, :, None], -math.inf)
    scores.masked_fill_((i >= count[:, None])[:, None, :, None, None], -math.inf)
    p = scores.sub_(scores.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp(min=1e-38))
    out = None
    if with_out:
        v = s["v_cache"][table].view(n, -1, hkv, d)[:, :length].float()
        v = v.masked_fill((j >= ctx[:, None])[:, :, None, None], 0.0).permute(0, 2, 1, 3)
        out = torch.matmul(p.view(n, hkv, g, length), v).reshape(n, hq, d).to(query.dtype)
    return p.sum((2, 3)), out


def _add_weights(s, c, added, fresh):
    """weights = decay * weights + added over each context; the last `fresh` tokens' own start here."""
    j = torch.arange(s["max_ctx"], device=added.device)
    ctx = s["context_lens"].long()[:, None, None]
    old = s["weights"][:, :, :s["max_ctx"]]
    faded = old * c["decay"] if c["decay"] else torch.zeros_like(old)
    new = torch.where(j < ctx - fresh.long()[:, None, None], faded, 0.0) + added
    old.copy_(torch.where(j < ctx, new, old))


def _evicted(s, c):
    n, hkv, d, bs, most = c["seqs"], c["kv_heads"], c["dim"], c["block"], c["keep"]
    length = s["max_ctx"]
    dev = s["weights"].device
    j = torch.arange(length, device=dev)
    ctx = s["context_lens"].long()[:, None, None]
    keep = torch.minimum(s["keep_lens"].long()[:, None, None], ctx)
    recent = keep.clamp(max=c["recent"])
    sinks = torch.minimum(keep - recent, torch.full_like(keep, c["sinks"]))
    w = s["weights"][:, :, :length]
    # first and last tokens ahead of the others, those by weight, equal ones by position
    group = torch.where((j < sinks) | (j >= ctx - recent), 0, 1).masked_fill(j >= ctx, 2).expand(n, hkv, length)
    order = w.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, group.gather(-1, order).sort(dim=-1, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, j.expand(n, hkv, length))
    kept = torch.where(rank < keep, j, length).sort(-1).values[:, :, :most]
    live = torch.arange(kept.shape[-1], device=dev) < keep
    at = kept.clamp(max=length - 1)
    s["kept"][:, :, :kept.shape[-1]] = torch.where(live, kept.int(), s["kept"][:, :, :kept.shape[-1]])
    to = s["new_weights"][:, :, :kept.shape[-1]]
    to.copy_(torch.where(live, w.gather(-1, at), to))
    b, h, i = live.expand(n, hkv, -1).nonzero(as_tuple=True)
    src = at[b, h, i]
    old_slot = s["block_tables"].long()[b, src // bs] * bs + src % bs
    new_slot = s["new_tables"].long()[b, i // bs] * bs + i % bs
    for cache in (s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)):
        cache[new_slot, h] = cache[old_slot, h]
    return s["kept"], s["new_weights"], s["k_cache"], s["v_cache"]


def _counted(s, c):
    """(first query row, query rows) of each sequence that count, and the most of any."""
    q_len = s["query_start"].diff().long()
    count = q_len.clamp(max=c["window"]) if c["window"] else q_len
    most = min(s["max_q"], c["window"]) if c["window"] else s["max_q"]
    return s["query_start"][1:].long() - count, count, most


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import paged_kv_cache_121_gb300 as pa
        layout = pa.PA_ROPE_INTERLEAVED if c.get("interleaved") else pa.PA_ROPE_HALF
        if op == "norm_rope":
            pa.pa_norm_rope(s["out"], s["x"], s["weight"], s["eps"], s["positions"], s["inv_freq"], layout=layout)
            return s["out"]
        if op == "norm_rope_grad":
            pa.pa_norm_rope_backward(s["grad_x"], s["grad_weight"], s["grad_out"], s["x"], s["weight"], s["eps"],
                                     s["positions"], s["inv_freq"], s["workspace"], layout=layout)
            return s["grad_x"], s["grad_weight"]
        if op == "norm_rope_cache":
            pa.pa_norm_rope_and_cache(s["query_out"], s["query"], s["key"], s["value"], s["query_weight"], s["key_weight"],
                                      s["eps"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["inv_freq"],
                                      layout=layout)
            return s["query_out"], s["k_cache"], s["v_cache"]
        if op == "decode_weights":
            pa.pa_decode_weights(s["out"], s["weights"], s["query"], s["k_cache"], s["v_cache"], s["block_tables"],
                                 s["context_lens"], s["max_ctx"], s["scale"], s["workspace"], decay=c["decay"])
            return s["out"], s["weights"]
        if op == "prefill_weights":
            pa.pa_prefill_weights(s["weights"], s["query"], s["k_cache"], s["block_tables"], s["context_lens"],
                                  s["query_start"], s["max_q"], s["max_ctx"], s["scale"], s["workspace"], decay=c["decay"],
                                  window=c["window"])
            return s["weights"]
        pa.pa_evict(s["kept"], s["new_weights"], s["weights"], s["k_cache"], s["v_cache"], s["block_tables"],
                    s["context_lens"], s["new_tables"], s["keep_lens"], s["max_ctx"], sinks=c["sinks"], recent=c["recent"])
        return s["kept"], s["new_weights"], s["k_cache"], s["v_cache"]
    if op == "norm_rope":
        y = _rotated(_normed(s["x"], s["weight"], s["eps"]), _turn(s, c), c["rot"], c["interleaved"])
        s["out"].copy_(y)
        return s["out"]
    if op == "norm_rope_grad":
        grad_x, grad_weight = _norm_rope_grad(s, c)
        s["grad_x"].copy_(grad_x)
        s["grad_weight"].copy_(grad_weight)
        return s["grad_x"], s["grad_weight"]
    if op == "norm_rope_cache":
        turn, padding = _turn(s, c), (s["positions"] < 0)[:, None, None]
        q = _rotated(_normed(s["query"], s["query_weight"], s["eps"]), turn, c["rot"], c["interleaved"])
        s["query_out"].copy_(torch.where(padding, s["query_out"].float(), q))
        hkv, d = c["kv_heads"], c["dim"]
        k, v = s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)
        # padding tokens are the last ones: the tokens before them have distinct slots
        live = c["tokens"] - c["padding"]
        slots = s["slots"][:live]
        y = _rotated(_normed(s["key"], s["key_weight"], s["eps"]), turn, c["rot"], c["interleaved"])
        k[slots] = y[:live].to(k.dtype)
        v[slots] = s["value"][:live]
        return s["query_out"], s["k_cache"], s["v_cache"]
    if op == "decode_weights":
        one = torch.ones_like(s["context_lens"]).long()
        added, out = _attended(s, c, s["query_start"][:-1].long(), one, 1, True)
        _add_weights(s, c, added, one)
        s["out"].copy_(out)
        return s["out"], s["weights"]
    if op == "prefill_weights":
        added, _ = _attended(s, c, *_counted(s, c), False)
        _add_weights(s, c, added, s["query_start"].diff())
        return s["weights"]
    return _evicted(s, c)


# --------------------------------------------------------------------------
# work, and the definition in 64 bits
# --------------------------------------------------------------------------
def work(case):
    e, d, op = BYTES[case["dtype"]], case["dim"], case["op"]
    if op in ("norm_rope", "norm_rope_grad"):
        t, h = case["tokens"], case["heads"]
        moved = (2 if op == "norm_rope" else 3) * t * h * d * e
        return dict(bytes=moved + 4 * t + 4 * case["rot"] + d * e, flops=t * h * ((4 if op == "norm_rope" else 9) * d + 3 * case["rot"]))
    if op == "norm_rope_cache":
        t, hq, hkv = case["tokens"] - case["padding"], case["heads"], case["kv_heads"]
        return dict(bytes=2 * t * (hq + 2 * hkv) * d * e + 12 * case["tokens"] + 4 * case["rot"] + 2 * d * e,
                    flops=t * (hq + hkv) * (4 * d + 3 * case["rot"]))
    q, ctx = _lens(case)
    hkv, n = case["kv_heads"], case["seqs"]
    table = 4 * int((-(-ctx // case["block"])).sum())
    if op == "evict":
        keep = np.minimum(ctx, case["keep"])
        kept = int(keep.sum()) * hkv
        return dict(bytes=kept * (4 * d * e + 8) + int(ctx.sum()) * hkv * 4 + table + 8 * n, flops=int(ctx.sum()) * hkv)
    hq = case["heads"]
    weights = 8 * int(ctx.sum()) * hkv
    if op == "decode_weights":
        return dict(bytes=2 * n * hq * d * e + 2 * int(ctx.sum()) * hkv * d * e + weights + table + 4 * n,
                    flops=4 * d * hq * int(ctx.sum()))
    w = np.minimum(q, case["window"]) if case["window"] else q
    pairs = int((w * (ctx - w) + w * (w + 1) // 2).sum())   # token i of the last w sees ctx - w + i + 1 tokens
    return dict(bytes=int(w.sum()) * hq * d * e + int(ctx.sum()) * hkv * d * e + weights + table + 8 * n,
                flops=2 * d * hq * pairs)


def exact(case, seed):
    if case["op"] == "evict":
        return None   # nothing is computed: tokens are chosen and moved
    s = prepare(case, seed)
    op, d = case["op"], case["dim"]
    if op.startswith("norm_rope"):
        half = case["rot"] // 2
        theta = torch.outer(s["positions"].double(), s["inv_freq"])
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)

        def turned(y, sign):   # a pair is a complex number, turned by e^(i theta)
            y = y.clone()
            z = torch.complex(y[:, :, first], y[:, :, second]) * torch.polar(torch.ones_like(theta), sign * theta)[:, None]
            y[:, :, first], y[:, :, second] = z.real, z.imag
            return y

        def unit(x):
            return x.double() / torch.sqrt((x.double() ** 2).sum(-1, keepdim=True) / d + s["eps"])

        if op == "norm_rope":
            return turned(unit(s["x"]) * s["weight"].double(), 1)
        if op == "norm_rope_grad":
            x = s["x"].double().requires_grad_()
            w = s["weight"].double().requires_grad_()
            y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + s["eps"]) * w
            return torch.autograd.grad(y, (x, w), turned(s["grad_out"].double(), -1))
        live = case["tokens"] - case["padding"]
        q = s["query_out"].double()
        q[:live] = turned(unit(s["query"]) * s["query_weight"].double(), 1)[:live]
        k, v = s["k_cache"].double(), s["v_cache"].double()
        block, offset = s["slots"][:live] // case["block"], s["slots"][:live] % case["block"]
        k[block, offset] = turned(unit(s["key"]) * s["key_weight"].double(), 1)[:live]
        v[block, offset] = s["value"][:live].double()
        return q, k, v
    q_lens, ctx = _lens(case)
    hq, hkv = case["heads"], case["kv_heads"]
    weights = s["weights"].double()
    out = torch.zeros(case["seqs"], hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["seqs"]):
        n, length = int(q_lens[b]), int(ctx[b])
        count = min(n, case["window"]) if case.get("window") else n
        where = torch.arange(length, device="cuda")
        blocks = s["block_tables"][b].long()[where // case["block"]]
        k, v = (s[c][blocks, where % case["block"]].double() for c in ("k_cache", "v_cache"))
        at += n
        hidden = torch.ones(count, length, dtype=torch.bool, device="cuda").triu(length - count + 1)
        weights[b, :, :length] *= case["decay"]
        weights[b, :, length - n:length] = 0
        for h in range(hq):
            g = h // (hq // hkv)
            logits = s["query"][at - count:at, h].double() @ k[:, g].T * s["scale"]
            p = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
            weights[b, g, :length] += p.sum(0)
            if op == "decode_weights":
                out[b, h] = p[0] @ v[:, g]
    return (out, weights) if op == "decode_weights" else weights
