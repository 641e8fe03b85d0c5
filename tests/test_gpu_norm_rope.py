"""pa_norm_rope, pa_norm_rope_and_cache and pa_norm_rope_backward against the
norm, the rotation and their derivatives in 64 bits.

Tolerances, derived. Let e = 2^-24 (half a step of fp32).
  Forward: the sum of D squares has at most log2 and serial roundings, under
  D e relative in any order (all terms positive); rsqrt is good to 2 units (4 e);
  the products by r and w round twice. So y = w x r is off by less than
  (D / 2 + 8) e |y|, and a rotated element by that of both of its pair's
  elements, plus the 8 e (|a| + |b|) of the angle and the rotation (derived in
  test_gpu_rope.py); then half a step of the output's type.
  Gradients: g (a rotation: 8 e of |ga| + |gb|) times w and u round three times
  more; the mean of D products of both signs is off by less than D e times the
  mean of their magnitudes. So dx = r (w g - u m) is off by less than
  (2 D + 32) e times r (|w| G + |u| mean|w G u|), G the pair's |ga| + |gb|, and
  half a step. dw sums N products, each off by less than (D + 32) e |G u|, in any
  order: under (N + D + 32) e times the sum of magnitudes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from test_gpu_rope import DT, SHAPES, rotate64

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
EPS = 1e-6


def half_step(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs() + 2.0 ** -25 * (dtype == torch.float16)


def case(shape, dt, seed, big=3.0):
    T, H, D, rot = shape
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, D, generator=g) * big).to(dt)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(dt)
    pos = torch.from_numpy(np.random.default_rng(seed).integers(0, 131072, T).astype(np.int32))
    f = torch.from_numpy(pa.pa_rope_frequencies(rot, 1e4)[0])
    return x, w, pos, f, pos.double()[:, None] * f[None]


def forward64(x, w, angle, interleaved, factor):
    x, w = x.double(), w.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return rotate64(y, angle, interleaved, factor)


def check_forward(got, want, size, D, factor):
    tol = (D / 2 + 16) * E * size * max(factor, 1.0) * 2
    tol = tol + half_step(want.abs() + tol, got.dtype)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES + [(2, 3, 250, 250), (3, 2, 255, 6)])
def test_norm_rope_matches_64_bits(dt, interleaved, shape):
    T, H, D, rot = shape
    x, w, pos, f, angle = case(shape, DT[dt], 3)
    factor = 1.25 if T % 2 else 1.0
    want, size = forward64(x, w, angle, interleaved, factor)
    out = torch.full((T, H, D), float("nan"), dtype=DT[dt], device="cuda")
    xd, wd, pd, fd = x.cuda(), w.cuda(), pos.cuda(), f.cuda()
    pa.pa_norm_rope(out, xd, wd, EPS, pd, fd, layout=int(interleaved), factor=factor)
    check_forward(out, want, size, D, factor)
    pa.pa_norm_rope(xd, xd, wd, EPS, pd, fd, layout=int(interleaved), factor=factor)
    assert torch.equal(xd, out)     # in place


def grads64(x, w, go, angle, interleaved, factor):
    """(dx, its scale of error, dw, its scale) in 64 bits, from the formulas."""
    x, w = x.double(), w.double()
    D = x.shape[-1]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    u = x * r
    g, size = rotate64(go.double(), angle, interleaved, factor, True)
    size = size * max(factor, 1.0)
    dx = r * (w * g - u * (w * g * u).mean(-1, keepdim=True))
    sx = r * (w.abs() * size + u.abs() * (w.abs() * size * u.abs()).mean(-1, keepdim=True))
    return dx, (2 * D + 32) * E * sx, (g * u).sum((0, 1)), (x.shape[0] * x.shape[1] + D + 32) * E * (size * u.abs()).sum((0, 1))


def backward(go, x, w, pos, f, interleaved, factor, grad_x=None):
    T, H, D = x.shape
    gx = torch.full((T, H, D), float("nan"), dtype=x.dtype, device="cuda") if grad_x is None else grad_x
    gw = torch.full((D,), float("nan"), device="cuda")
    ws = torch.full((max(1, pa.pa_norm_rope_backward_workspace_size(T, H, D)),), 255, dtype=torch.uint8, device="cuda")
    pa.pa_norm_rope_backward(gx, gw, go, x, w, EPS, pos, f, ws, layout=int(interleaved), factor=factor)
    return gx, gw


def check_grads(gx, gw, want):
    dx, tx, dw, tw = want
    err = (gx.double().cpu() - dx).abs()
    tol = tx + half_step(dx.abs() + tx, gx.dtype)
    assert bool((err <= tol).all()), float((err - tol).max())
    err = (gw.double().cpu() - dw).abs()
    assert bool((err <= tw + half_step(dw.abs() + tw, torch.float32)).all()), float((err - tw).max())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES + [(2, 3, 250, 250), (3, 2, 255, 6)])
def test_gradients_match_64_bits(dt, interleaved, shape):
    T, H, D, rot = shape
    x, w, pos, f, angle = case(shape, DT[dt], 4)
    factor = 1.25 if T % 2 else 1.0
    go = torch.randn(T, H, D, generator=torch.Generator().manual_seed(5)).to(DT[dt])
    want = grads64(x, w, go, angle, interleaved, factor)
    god, xd, wd, pd, fd = go.cuda(), x.cuda(), w.cuda(), pos.cuda(), f.cuda()
    gx, gw = backward(god, xd, wd, pd, fd, interleaved, factor)
    check_grads(gx, gw, want)
    # in place of either operand, and the same bits again
    for t in (god.clone(), xd.clone()):
        args = (t, xd) if t.data_ptr() != 0 and torch.equal(t, god) else (god, t)
        a, b = backward(args[0], args[1], wd, pd, fd, interleaved, factor, grad_x=t)
        assert torch.equal(a, gx) and torch.equal(b, gw)


def test_gradients_against_differences():
    """The formulas of grads64 themselves: central differences of the 64-bit forward pass."""
    T, H, D, rot = shape = (2, 2, 10, 6)
    x, w, pos, f, angle = case(shape, torch.float64, 6, big=1.0)
    go = torch.randn(T, H, D, generator=torch.Generator().manual_seed(7)).double()

    def loss(x, w):
        return float((forward64(x, w, angle, False, 1.25)[0] * go).sum())

    dx, _, dw, _ = grads64(x, w, go, angle, False, 1.25)
    h = 1e-6
    for t, d in ((x, dx), (w, dw)):
        flat, df = t.view(-1), d.reshape(-1)
        for i in range(flat.numel()):
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss(x, w)
            flat[i] = keep - h
            down = loss(x, w)
            flat[i] = keep
            # central differences: h^2 times a third derivative of order 10, and roundings of 2^-53 |loss| / h
            assert abs((up - down) / (2 * h) - float(df[i])) <= 1e-7


@pytest.mark.parametrize("dt", list(DT))
def test_views_padding_and_odd_alignment(dt):
    """Heads of a wider, shifted row; padding tokens keep what the outputs held, and count for nothing."""
    T, H, D, rot = shape = (37, 5, 64, 32)
    x, w, pos, f, angle = case(shape, DT[dt], 8)
    pos[[0, 5, 36]] = -1
    live = pos >= 0
    x[~live] = float("nan")
    go = torch.randn(T, H, D, generator=torch.Generator().manual_seed(9)).to(DT[dt])
    go[~live] = float("inf")

    def wide(t, shift):   # rows 7 elements wider, starting `shift` elements in
        buf = torch.full((T * (H * D + 7) + shift,), 3.0, dtype=DT[dt], device="cuda")
        v = buf[shift:].view(T, H * D + 7)[:, :H * D].view(T, H, D)
        v.copy_(t)
        return v

    for shift in (0, 1, 2):
        xd, god = wide(x, shift), wide(go, shift)
        out, gx = wide(torch.full_like(x, 3.0), shift), wide(torch.full_like(x, 3.0), shift)
        wd = torch.cat([w[:shift], w]).cuda()[shift:]
        pa.pa_norm_rope(out, xd, wd, EPS, pos.cuda(), f.cuda())
        want, size = forward64(x[live], w, angle[live], False, 1.0)
        check_forward(out.cpu()[live], want, size, D, 1.0)
        gw = torch.empty(D, device="cuda")
        ws = torch.empty(pa.pa_norm_rope_backward_workspace_size(T, H, D), dtype=torch.uint8, device="cuda")
        pa.pa_norm_rope_backward(gx, gw, god, xd, wd, EPS, pos.cuda(), f.cuda(), ws)
        check_grads(gx.cpu()[live], gw, grads64(x[live], w, go[live], angle[live], False, 1.0))
        assert bool((out.cpu()[~live] == 3.0).all()) and bool((gx.cpu()[~live] == 3.0).all())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T", [1, 3, 700])
def test_append_is_norm_rope_then_the_scatter(dt, T):
    H, hkv, D, rot, bs = 12, 4, 128, 64, 16
    g = torch.Generator().manual_seed(T)
    qkv = (torch.randn(T, H + 2 * hkv, D, generator=g) * 2).to(DT[dt]).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + hkv], qkv[:, H + hkv:]
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(DT[dt]).cuda() for _ in range(2))
    rng = np.random.default_rng(T)
    pos = torch.from_numpy(rng.integers(0, 5000, T).astype(np.int32))
    blocks = -(-T // bs) + 2
    slots = torch.from_numpy(rng.permutation(blocks * bs)[:T].astype(np.int64))
    if T > 2:
        pos[1], slots[2] = -1, -5          # padding; a token without a slot (its query is rotated all the same)
    f = torch.from_numpy(pa.pa_rope_frequencies(rot, 1e6)[0]).cuda()
    kc, vc = (torch.randn(blocks, bs, hkv, D, generator=g).to(DT[dt]).cuda() for _ in range(2))
    kc0, vc0 = kc.clone(), vc.clone()
    qo = torch.full((T, H, D), 7.0, dtype=DT[dt], device="cuda")
    pa.pa_norm_rope_and_cache(qo, q, k, v, qw, kw, EPS, kc, vc, slots.cuda(), pos.cuda(), f)
    want_q = torch.full_like(qo, 7.0)
    pa.pa_norm_rope(want_q, q, qw, EPS, pos.cuda(), f)
    want_k = torch.empty(T, hkv, D, dtype=DT[dt], device="cuda")
    pa.pa_norm_rope(want_k, k, kw, EPS, pos.cuda(), f)
    masked = torch.where(pos >= 0, slots, torch.full_like(slots, -1)).cuda()
    pa.pa_reshape_and_cache(want_k, v.contiguous(), kc0, vc0, masked)
    assert torch.equal(qo, want_q) and torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_rows_of_zeros_and_no_tokens():
    x = torch.zeros(3, 2, 64, device="cuda")
    w, pos = torch.ones(64, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    f = torch.from_numpy(pa.pa_rope_frequencies(64, 1e4)[0]).cuda()
    out = torch.full_like(x, 9.0)
    pa.pa_norm_rope(out, x, w, EPS, pos, f)
    assert bool((out == 0).all())
    go = torch.ones_like(x)
    gx, gw = backward(go, x, w, pos, f, False, 1.0)
    want = grads64(x.cpu(), w.cpu(), go.cpu(), pos.cpu().double()[:, None] * f.cpu()[None], False, 1.0)
    check_grads(gx, gw, want)
    gw.fill_(5.0)
    none = x[:0]
    pa.pa_norm_rope_backward(none, gw, none, none, w, EPS, pos[:0], f, torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert bool((gw == 0).all())


def test_captured_and_replayed():
    T, H, D, rot = shape = (33, 8, 128, 128)
    x, w, pos, f, angle = case(shape, torch.bfloat16, 11)
    go = torch.randn(T, H, D, generator=torch.Generator().manual_seed(12)).bfloat16()
    xd, god, wd, pd, fd = x.cuda(), go.cuda(), w.cuda(), pos.cuda(), f.cuda()
    want_out = torch.empty_like(xd)
    pa.pa_norm_rope(want_out, xd, wd, EPS, pd, fd)
    want = backward(god, xd, wd, pd, fd, False, 1.0)
    out, gx, gw = torch.empty_like(xd), torch.empty_like(xd), torch.empty(D, device="cuda")
    ws = torch.empty(pa.pa_norm_rope_backward_workspace_size(T, H, D), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_norm_rope(out, xd, wd, EPS, pd, fd)
        pa.pa_norm_rope_backward(gx, gw, god, xd, wd, EPS, pd, fd, ws)
    for _ in range(3):
        out.zero_(), gx.zero_(), gw.zero_()
        graph.replay()
        assert torch.equal(out, want_out) and torch.equal(gx, want[0]) and torch.equal(gw, want[1])
