"""pa_prefill and pa_cross_attention, host side (CPU): what is refused returns
before any launch."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa

P = 4096   # a made-up, aligned address: no refused call touches it


def prefill(out=P, od=1, q=P, qd=1, k=P, v=P, kd=1, bt=P, cl=P, qs=P, B=2, T=8, hq=8, hkv=2, d=128, bs=16, mb=4, nb=9,
            mq=6, mc=64, scale=0.1, causal=1, ws=None, wsb=0):
    return pa.load_library().pa_prefill(out, od, q, qd, k, v, kd, bt, cl, qs, B, T, hq, hkv, d, bs, mb, nb, mq, mc,
                                        scale, causal, ws, wsb, None)


def cross(out=P, od=1, q=P, qd=1, k=P, v=P, kd=1, cl=P, qs=P, B=2, T=8, hq=8, hkv=2, d=128, states=64, mq=6, mc=64,
          scale=0.1, ws=None, wsb=0):
    return pa.load_library().pa_cross_attention(out, od, q, qd, k, v, kd, cl, qs, B, T, hq, hkv, d, states, mq, mc,
                                                scale, ws, wsb, None)


@pytest.mark.parametrize("call", [prefill, cross])
def test_nothing_to_do(call):
    assert call(B=0) == call(T=0) == call(mq=0) == pa.PA_OK


COMMON = [dict(out=None), dict(q=None), dict(k=None), dict(v=None), dict(cl=None), dict(qs=None), dict(B=-1),
          dict(T=-1), dict(mq=-1), dict(mc=-1), dict(hq=0), dict(hkv=0), dict(hq=9), dict(od=5), dict(qd=9, kd=9),
          dict(scale=float("nan")), dict(scale=float("inf")), dict(mc=65), dict(out=P + 8), dict(q=P + 2),
          dict(k=P + 4), dict(v=P + 8), dict(cl=P + 2), dict(qs=P + 1)]


@pytest.mark.parametrize("call", [prefill, cross])
@pytest.mark.parametrize("kw", COMMON, ids=str)
def test_invalid_arguments(call, kw):
    assert call(**kw) == pa.PA_ERR_INVALID_ARG


def test_invalid_pages():
    for kw in (dict(bt=None), dict(bt=P + 2), dict(bs=0), dict(mb=0), dict(nb=0)):
        assert prefill(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert cross(states=0) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [prefill, cross])
def test_unsupported(call):
    assert call(d=96) == call(d=256) == pa.PA_ERR_UNSUPPORTED
    assert call(qd=1, kd=2) == call(qd=0, kd=1) == pa.PA_ERR_UNSUPPORTED


def test_unsupported_sizes():
    assert prefill(bs=512) == pa.PA_ERR_UNSUPPORTED
    assert cross(B=1 << 16, states=1 << 16) == pa.PA_ERR_UNSUPPORTED


def test_binding_refuses_mismatched_tensors():
    q = torch.zeros(8, 8, 64)
    k = torch.zeros(9, 16, 2, 64)
    bt, cl, qs = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)

    def call(out=q, query=q, kc=k, vc=k, tables=bt, lens=cl, start=qs):
        pa.pa_prefill(out, query, kc, vc, tables, lens, start, 4, 64, 0.1)

    with pytest.raises(ValueError):
        call()                                   # not on a CUDA device
    for kw in (dict(out=torch.zeros(8, 8, 32)), dict(vc=torch.zeros(9, 16, 2, 32)), dict(start=qs[:2])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(query=q.half(), out=q.half()), dict(vc=k.half()), dict(lens=cl.long()), dict(start=qs.long())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(ValueError):
        pa.pa_cross_attention(q, q, k[:2], k[:1], cl, qs, 4, 16, 0.1)
