"""pa_rope and pa_rope_and_cache against the rotation in 64 bits.

Tolerance, derived: the kernel rounds the reduced angle to fp32 (half turns
in [-1, 1): at most 2^-25 of it, so pi 2^-25 of the angle), sincospif is good
to 2 units of 2^-24, the factor and the two products and their sum round once
each (2^-25 of at most |a| + |b| a piece): under 8 * 2^-24 * factor * (|a| +
|b|) in all. Then one rounding to the output's type: half a step,
eps / 2 * |y|, of the unrounded value (2^-25 below fp16's normal range)."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SHAPES = [  # tokens, heads, head_dim, rotary_dim
    (1, 1, 64, 64), (7, 5, 128, 64), (33, 40, 128, 128), (5, 3, 96, 40), (4, 2, 10, 6), (3, 2, 256, 256),
    (300, 11, 64, 16), (2, 1, 2, 2), (1201, 48, 128, 128),
]


def rotate64(x, angle, interleaved, factor=1.0, transpose=False):
    """x [T, H, D] float64, angle [T, rot/2] float64 -> (rotated, |a| + |b| of each element's pair)."""
    half = angle.shape[1]
    y, size = x.clone(), x.abs()
    i = torch.arange(half)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., a_at], x[..., b_at]
    c, s = angle.cos()[:, None] * factor, angle.sin()[:, None] * factor
    if transpose:
        s = -s
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    size[..., a_at] = size[..., b_at] = a.abs() + b.abs()
    return y, size


def close(got, want, size, factor=1.0):
    eps = torch.finfo(got.dtype).eps
    tol = eps / 2 * want.abs() * (1 + eps) + 8 * 2.0 ** -24 * factor * size * (1 + eps) + 2.0 ** -25 * (got.dtype == torch.float16)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def draw(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dt)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope_matches_64_bits(dt, interleaved, shape):
    T, H, D, rot = shape
    x = draw((T, H, D), DT[dt], 1)
    pos = torch.from_numpy(np.random.default_rng(2).integers(0, 131072, T).astype(np.int32))
    freq, _ = pa.pa_rope_frequencies(rot, 1e4)
    factor = 1.25 if T % 2 else 1.0
    f = torch.from_numpy(freq)
    angle = pos.double()[:, None] * f[None]
    for transpose in (False, True):
        want, size = rotate64(x.double(), angle, interleaved, factor, transpose)
        xd, out = x.cuda(), torch.full((T, H, D), float("nan"), dtype=DT[dt], device="cuda")
        pa.pa_rope(out, xd, pos.cuda(), f.cuda(), layout=int(interleaved), factor=factor, transpose=transpose)
        close(out, want, size, factor)
        assert torch.equal(out[..., rot:].cpu(), x[..., rot:])     # past the rotated part: bit for bit
        pa.pa_rope(xd, xd, pos.cuda(), f.cuda(), layout=int(interleaved), factor=factor, transpose=transpose)
        assert torch.equal(xd, out)                                # in place


def test_far_positions_are_exact():
    """Positions up to 2^31 - 1 and below zero's neighbours: the angle reduced modulo a turn with 60 digits."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    T, D = 6, 128
    pos = np.array([0, 1, 65537, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1], np.int32)
    freq, _ = pa.pa_rope_frequencies(D, 1e6)
    freq[3], freq[5] = -freq[3], 5.75      # any frequency may be passed
    angle = torch.tensor([[float((Decimal(int(p)) * Decimal(float(f))) % two_pi) for f in freq] for p in pos],
                         dtype=torch.float64)
    x = draw((T, 3, D), torch.float32, 3)
    for interleaved in (0, 1):
        want, size = rotate64(x.double(), angle, bool(interleaved))
        out = torch.empty_like(x, device="cuda")
        pa.pa_rope(out, x.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), layout=interleaved)
        close(out, want, size)


def test_transpose_is_the_gradient():
    """<R x, g> = <x, R^T g>, and central differences of <R x, g> in x give R^T g (R is linear in x,
    so the difference quotient has no truncation error: what is left are the roundings)."""
    T, H, D = 5, 2, 64
    x, g = draw((T, H, D), torch.float32, 4), draw((T, H, D), torch.float32, 5)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 999
    f = torch.from_numpy(pa.pa_rope_frequencies(D, 1e4)[0]).cuda()

    def rot(v, transpose=False):
        out = torch.empty(T, H, D, device="cuda")
        pa.pa_rope(out, v.cuda(), pos, f, layout=1, factor=1.5, transpose=transpose)
        return out.double().cpu()

    back = rot(g, transpose=True)
    # 2 D T H terms, each of relative size 8 * 2^-24 at most
    lhs, rhs = (rot(x) * g.double()).sum(), (x.double() * back).sum()
    assert abs(lhs - rhs) <= 8 * 2.0 ** -24 * 1.5 * 2 * float((x.abs().double() * 2).sum() * g.abs().max())
    for t, h, d in ((0, 0, 0), (2, 1, 33), (4, 0, 63)):
        step = torch.zeros_like(x)
        step[t, h, d] = 1.0
        quotient = ((rot(x + step) - rot(x - step)) * g.double()).sum() / 2
        size = float((x.abs() + 1)[t, h].sum() * 2)     # only that head's outputs differ
        assert abs(quotient - back[t, h, d]) <= 16 * 2.0 ** -24 * 1.5 * size * float(g.abs().max())


@pytest.mark.parametrize("offset", [0, 1, 2])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rope_on_strided_views(dt, offset):
    """Token rows further apart than a head list, from bases that are 16-byte aligned or not."""
    T, H, D, wide = 9, 4, 64, 4 * 64 + 64 + 8 * offset
    flat = draw((T * wide + 16,), DT[dt], 6).cuda()
    x = flat.as_strided((T, H, D), (wide, D, 1), offset)
    dst = torch.full_like(flat, 7.0)
    out = dst.as_strided((T, H, D), (wide, D, 1), offset)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 31
    f = torch.from_numpy(pa.pa_rope_frequencies(D, 1e4)[0]).cuda()
    pa.pa_rope(out, x, pos, f)
    want, size = rotate64(x.double().cpu(), pos.double().cpu()[:, None] * f.cpu()[None], False)
    close(out, want, size)
    mask = torch.ones_like(flat, dtype=torch.bool)
    mask.as_strided((T, H, D), (wide, D, 1), offset).fill_(False)
    assert bool((dst[mask] == 7.0).all())         # nothing between the rows is written


def test_padding_and_empty():
    T, H, D = 11, 3, 128
    x = draw((T, H, D), torch.bfloat16, 7).cuda()
    pos = torch.tensor([5, -1, 7, -2 ** 31, 0, 1, 2, 3, -5, 9, -1], dtype=torch.int32, device="cuda")
    f = torch.from_numpy(pa.pa_rope_frequencies(D, 1e4)[0]).cuda()
    out = torch.full_like(x, 9.0)
    pa.pa_rope(out, x, pos, f)
    dead = pos < 0
    assert bool((out[dead] == 9.0).all()) and not bool((out[~dead] == 9.0).all())
    pa.pa_rope(out[:0], x[:0], pos[:0], f)        # no tokens


def append_case(T, hq, hkv, D, rot, bs, dt, interleaved, seed, fused=True):
    rng = np.random.default_rng(seed)
    qkv = draw((T, hq + 2 * hkv, D), DT[dt], seed).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = -(-T // bs) + 3
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    pos = rng.integers(0, 100000, T).astype(np.int32)
    if T > 4:
        slots[1], slots[3], pos[2] = -1, nb * bs + 5, -4     # no slot, a slot past the pool, padding
    caches = [draw((nb, bs, hkv, D), DT[dt], seed + 1 + i).cuda() for i in range(2)]
    f = torch.from_numpy(pa.pa_rope_frequencies(rot, 1e4, pa.PA_ROPE_YARN, 4.0, 4096)[0]).cuda()
    return q, k, v, caches[0], caches[1], torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), f


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dims", [(1, 4, 2, 128, 128, 16), (16, 32, 8, 128, 128, 16), (77, 6, 3, 64, 32, 1),
                                  (900, 8, 8, 128, 64, 32), (13, 5, 1, 96, 40, 12), (6, 2, 2, 20, 12, 8)])
def test_append_matches_64_bits_and_separate_calls(dt, interleaved, dims):
    T, hq, hkv, D, rot, bs = dims
    q, k, v, kc, vc, slots, pos, f = append_case(T, hq, hkv, D, rot, bs, dt, interleaved, 20)
    k0, v0 = kc.clone(), vc.clone()
    qo = torch.full((T, hq, D), 3.0, dtype=DT[dt], device="cuda")
    pa.pa_rope_and_cache(qo, q, k, v, kc, vc, slots, pos, f, layout=int(interleaved), factor=1.1)
    angle = pos.double().cpu()[:, None] * f.cpu()[None]
    live = (pos >= 0).cpu()
    want, size = rotate64(q.double().cpu(), angle, interleaved, 1.1)
    close(qo[live.cuda()], want[live], size[live], 1.1)
    assert bool((qo[~live.cuda()] == 3.0).all())
    # the same by pa_rope and pa_reshape_and_cache, bit for bit
    qo2 = torch.full_like(qo, 3.0)
    pa.pa_rope(qo2, q, pos, f, layout=int(interleaved), factor=1.1)
    kr = torch.zeros(T, hkv, D, dtype=DT[dt], device="cuda")
    pa.pa_rope(kr, k, pos, f, layout=int(interleaved), factor=1.1)
    wk, sk = rotate64(k.double().cpu(), angle, interleaved, 1.1)
    close(kr[live.cuda()], wk[live], sk[live], 1.1)
    pa.pa_reshape_and_cache(kr, v.contiguous(), k0, v0, torch.where(pos < 0, -torch.ones_like(slots), slots))
    assert torch.equal(qo, qo2) and torch.equal(kc, k0) and torch.equal(vc, v0)


def test_append_in_place_on_streams_and_in_a_graph():
    """query_out = query; another stream than the current one; captured and replayed with new inputs."""
    T, hq, hkv, D = 24, 8, 2, 128
    q, k, v, kc, vc, slots, pos, f = append_case(T, hq, hkv, D, D, 16, "bf16", False, 30, fused=False)
    want_q = torch.empty_like(q)
    wk, wv = kc.clone(), vc.clone()
    pa.pa_rope_and_cache(want_q, q, k, v, wk, wv, slots, pos, f)
    pad = pos < 0
    want_q[pad] = q[pad]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q2, k2, v2 = q.clone(), kc.clone(), vc.clone()
    torch.cuda.synchronize()
    pa.pa_rope_and_cache(q2, q2, k, v, k2, v2, slots, pos, f, stream=s)
    s.synchronize()
    assert torch.equal(q2, want_q) and torch.equal(k2, wk) and torch.equal(v2, wv)
    qo, k3, v3 = torch.zeros_like(q), kc.clone(), vc.clone()
    qi = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_rope_and_cache(qo, qi, k, v, k3, v3, slots, pos, f)
    qi.copy_(q)
    qo.copy_(q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want_q) and torch.equal(k3, wk) and torch.equal(v3, wv)


def test_append_far_slots():
    """Slots whose byte offset in the cache passes 2^32."""
    hkv, D, bs = 8, 128, 16
    nb = (1 << 32) // (bs * hkv * D * 2) + 64
    kc = torch.zeros(nb, bs, hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    T = 32
    q, k, v, _, _, _, pos, f = append_case(T, 8, hkv, D, D, bs, "bf16", False, 40)
    pos = pos.abs()
    slots = torch.arange(nb * bs - T, nb * bs, dtype=torch.int64, device="cuda")
    qo = torch.empty(T, 8, D, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_and_cache(qo, q, k, v, kc, vc, slots, pos, f)
    kr = torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope(kr, k, pos, f)
    assert torch.equal(kc.view(-1, hkv, D)[-T:], kr) and torch.equal(vc.view(-1, hkv, D)[-T:], v)
    assert not bool(kc.view(-1, hkv, D)[:-T].any())
