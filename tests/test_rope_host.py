"""Rotary positions, host side (CPU): the frequencies of every scaling kind
against their formulas, and the argument checks of pa_rope and
pa_rope_and_cache, which return before any launch."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa


def plain(r, base):
    return np.array([base ** (-2.0 * i / r) for i in range(r // 2)])


@pytest.mark.parametrize("r", [2, 6, 64, 128])
@pytest.mark.parametrize("base", [1e4, 1e6])
def test_frequencies_of_each_kind(r, base):
    f = plain(r, base)
    got, factor = pa.pa_rope_frequencies(r, base)
    assert np.allclose(got, f, rtol=1e-14) and factor == 1.0
    got, factor = pa.pa_rope_frequencies(r, base, pa.PA_ROPE_LINEAR, 4.0)
    assert np.allclose(got, f / 4, rtol=1e-14) and factor == 1.0
    if r > 2:
        got, factor = pa.pa_rope_frequencies(r, base, pa.PA_ROPE_NTK, 8.0)
        assert np.allclose(got, plain(r, base * 8 ** (r / (r - 2))), rtol=1e-13) and factor == 1.0
        # the slowest pair is slowed by the scale exactly, the fastest not at all
        assert got[0] == 1.0 and math.isclose(got[-1], f[-1] / 8, rel_tol=1e-12)
    got, factor = pa.pa_rope_frequencies(r, base, pa.PA_ROPE_BANDS, 8.0, 8192, 1.0, 4.0)
    for g, w in zip(got, f):
        turns = 8192 * w / (2 * math.pi)
        want = w if turns >= 4 else w / 8 if turns <= 1 else w / 8 * (4 - turns) / 3 + w * (turns - 1) / 3
        assert math.isclose(g, want, rel_tol=1e-12)
    assert factor == 1.0


def test_yarn_keeps_fast_pairs_and_interpolates_slow_ones():
    r, base, scale, ctx = 128, 1e4, 16.0, 4096
    f = plain(r, base)
    got, factor = pa.pa_rope_frequencies(r, base, pa.PA_ROPE_YARN, scale, ctx, 1.0, 32.0)
    assert factor == np.float32(0.1 * math.log(scale) + 1)
    first = math.floor(r * math.log(ctx / (32 * 2 * math.pi)) / (2 * math.log(base)))
    last = math.ceil(r * math.log(ctx / (1 * 2 * math.pi)) / (2 * math.log(base)))
    for i in range(r // 2):
        ramp = min(max((i - first) / (last - first), 0.0), 1.0)
        assert math.isclose(got[i], f[i] / scale * ramp + f[i] * (1 - ramp), rel_tol=1e-12)
    assert np.array_equal(got[: first + 1], pa.pa_rope_frequencies(r, base)[0][: first + 1])
    assert pa.pa_rope_frequencies(r, base, pa.PA_ROPE_YARN, 1.0, ctx)[1] == 1.0


@pytest.mark.parametrize("args", [
    (0, 1e4), (5, 1e4), (-2, 1e4), (64, 1.0), (64, float("nan")), (64, float("inf")),
    (64, 1e4, 9, 2.0), (64, 1e4, -1, 2.0), (64, 1e4, pa.PA_ROPE_LINEAR, 0.0), (2, 1e4, pa.PA_ROPE_NTK, 2.0),
    (64, 1e4, pa.PA_ROPE_YARN, 2.0, 0), (64, 1e4, pa.PA_ROPE_YARN, 2.0, 4096, 32.0, 1.0),
    (64, 1e4, pa.PA_ROPE_BANDS, float("nan"), 4096), (64, 1e4, pa.PA_ROPE_BANDS, 2.0, 4096, 0.0, 4.0),
])
def test_frequencies_refusals(args):
    with pytest.raises(pa.PAError) as e:
        pa.pa_rope_frequencies(*args)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_argument_checks_return_before_launch():
    lib = pa.load_library()
    P = 4096   # a made-up, aligned address: no refused call touches it

    def rope(out=P, so=512, x=P, sx=512, pos=P, f=P, T=4, H=4, D=128, rot=128, layout=0, factor=1.0, dtype=1):
        return lib.pa_rope(out, so, x, sx, pos, f, T, H, D, rot, layout, factor, 0, dtype, None)

    assert rope(T=0) == pa.PA_OK
    bad = [dict(out=None), dict(x=None), dict(pos=None), dict(f=None), dict(T=-1), dict(H=0), dict(D=0), dict(rot=0),
           dict(rot=3), dict(rot=130), dict(layout=2), dict(factor=float("nan")), dict(dtype=7), dict(so=511),
           dict(sx=511), dict(x=P + 1), dict(f=P + 4), dict(pos=P + 2)]
    for kw in bad:
        assert rope(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert rope(D=512, so=4096, sx=4096) == pa.PA_ERR_UNSUPPORTED

    def append(qo=P, sqo=512, q=P, sq=512, k=P, sk=256, v=P, sv=256, kc=P, vc=P, slots=P, pos=P, f=P, T=4, H=4, nb=8,
               bs=16, hkv=2, D=128, rot=128, layout=0, factor=1.0, dtype=1):
        return lib.pa_rope_and_cache(qo, sqo, q, sq, k, sk, v, sv, kc, vc, slots, pos, f, T, H, nb, bs, hkv, D, rot,
                                     layout, factor, dtype, None)

    assert append(T=0) == pa.PA_OK
    for name in ("qo", "q", "k", "v", "kc", "vc", "slots", "pos", "f"):
        assert append(**{name: None}) == pa.PA_ERR_INVALID_ARG, name
    for kw in (dict(nb=0), dict(bs=0), dict(hkv=0), dict(sk=255), dict(sv=255), dict(sqo=511), dict(kc=P + 8),
               dict(vc=P + 8), dict(slots=P + 4), dict(rot=129), dict(layout=-1), dict(factor=float("inf"))):
        assert append(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert append(hkv=1, D=6, rot=6) == pa.PA_ERR_UNSUPPORTED   # a slot is not whole 16-byte vectors


def test_in_place_needs_one_stride():
    """Rows rotated in place but at another stride would overwrite rows that are still to be read."""
    lib = pa.load_library()
    P = 4096
    assert lib.pa_rope(P, 1024, P, 512, P, P, 4, 4, 128, 128, 0, 1.0, 0, 1, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_rope_and_cache(P, 512, P, 768, P, 256, P, 256, P, P, P, P, P, 4, 4, 8, 16, 2, 128, 128, 0, 1.0, 1,
                                 None) == pa.PA_ERR_INVALID_ARG


def test_binding_refuses_mismatched_tensors():
    T, H, D = 4, 2, 64
    x = torch.zeros(T, H, D)
    pos = torch.zeros(T, dtype=torch.int32)
    f = torch.zeros(D // 2, dtype=torch.float64)
    with pytest.raises(ValueError):    # not on a CUDA device
        pa.pa_rope(torch.empty_like(x), x, pos, f)
    with pytest.raises(ValueError):    # shape
        pa.pa_rope(torch.empty(T, H, D + 2), x, pos, f)
    with pytest.raises(ValueError):    # dtype
        pa.pa_rope(torch.empty(T, H, D, dtype=torch.float16), x, pos, f)
    with pytest.raises(TypeError):
        pa.pa_rope(torch.empty_like(x), x, pos.long(), f)
    with pytest.raises(TypeError):
        pa.pa_rope(torch.empty_like(x), x, pos[:3], f)
    with pytest.raises(TypeError):
        pa.pa_rope(torch.empty_like(x), x, pos, f.float())
    cache = torch.zeros(8, 16, 1, D)
    slots = torch.zeros(T, dtype=torch.int64)
    k = torch.zeros(T, 1, D)
    with pytest.raises(TypeError):
        pa.pa_rope_and_cache(x.clone(), x, k, k, cache, cache.clone(), slots.int(), pos, f)
    with pytest.raises(TypeError):     # the query of another type than the caches
        pa.pa_rope_and_cache(x.half(), x.half(), k, k, cache, cache.clone(), slots, pos, f)
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache(x.clone(), x, k[:3], k, cache, cache.clone(), slots, pos, f)
