"""The calls around attention weights, host side (CPU): argument checks that return before any launch, the
binding's refusals, and the block manager's compaction."""
import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa

P = 4096   # a made-up, aligned address: no refused call touches it
NAN, INF = float("nan"), float("inf")


def test_norm_rope_checks_return_before_launch():
    lib = pa.load_library()

    def fwd(out=P, so=512, x=P, sx=512, w=P, eps=1e-6, pos=P, f=P, T=4, H=4, D=128, rot=128, layout=0, factor=1.0, dtype=1):
        return lib.pa_norm_rope(out, so, x, sx, w, eps, pos, f, T, H, D, rot, layout, factor, dtype, None)

    def bwd(gx=P, sg=512, gw=P, go=P, so=512, x=P, sx=512, w=P, eps=1e-6, pos=P, f=P, T=4, H=4, D=128, rot=128, layout=0,
            factor=1.0, dtype=1):
        return lib.pa_norm_rope_backward(gx, sg, gw, go, so, x, sx, w, eps, pos, f, T, H, D, rot, layout, factor, dtype, P,
                                         1 << 30, None)

    assert fwd(T=0) == pa.PA_OK
    common = [dict(x=None), dict(w=None), dict(pos=None), dict(f=None), dict(T=-1), dict(H=0), dict(D=0), dict(rot=0),
              dict(rot=3), dict(rot=130), dict(layout=2), dict(factor=NAN), dict(dtype=7), dict(so=511), dict(sx=511),
              dict(x=P + 1), dict(w=P + 1), dict(f=P + 4), dict(pos=P + 2), dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF)]
    for kw in common + [dict(out=None), dict(so=1024)]:   # (the last: in place at two strides)
        assert fwd(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in common + [dict(gx=None), dict(gw=None), dict(go=None), dict(sg=511), dict(sg=1024), dict(gw=P + 2)]:
        assert bwd(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert fwd(D=512, so=4096, sx=4096) == pa.PA_ERR_UNSUPPORTED

    def append(qw=P, kw=P, eps=1e-6, T=4, kc=P, D=128, rot=128, hkv=2):
        return lib.pa_norm_rope_and_cache(P, 512, P, 512, P, 256, P, 256, qw, kw, eps, kc, P, P, P, P, T, 4, 8, 16, hkv, D,
                                          rot, 0, 1.0, 1, None)

    assert append(T=0) == pa.PA_OK
    for kw in (dict(qw=None), dict(kw=None), dict(qw=P + 1), dict(eps=NAN), dict(eps=-1.0), dict(kc=P + 8), dict(hkv=0)):
        assert append(**kw) == pa.PA_ERR_INVALID_ARG, kw


def test_weights_checks_return_before_launch():
    lib = pa.load_library()

    def decode(out=P, odt=1, w=P, ws=128, q=P, qdt=1, k=P, v=P, kdt=1, bt=P, cl=P, B=2, hq=8, hkv=2, D=64, bs=16, mb=8,
               nb=20, mc=128, scale=0.1, decay=1.0, space=P, size=1 << 30):
        return lib.pa_decode_weights(out, odt, w, ws, q, qdt, k, v, kdt, bt, cl, B, hq, hkv, D, bs, mb, nb, mc, scale, decay,
                                     space, size, None)

    assert decode(B=0) == pa.PA_OK
    for kw in (dict(out=None), dict(w=None), dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(cl=None),
               dict(ws=127), dict(B=-1), dict(hq=7), dict(hkv=0), dict(mc=129), dict(scale=NAN), dict(decay=NAN),
               dict(decay=-0.5), dict(decay=INF), dict(odt=5), dict(qdt=9), dict(q=P + 8), dict(k=P + 2), dict(w=P + 2),
               dict(cl=P + 1)):
        assert decode(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(D=96), dict(bs=512, mc=128), dict(qdt=1, kdt=2), dict(B=70000)):
        assert decode(**kw) == pa.PA_ERR_UNSUPPORTED, kw
    for kw in (dict(space=None), dict(size=8 * 2 * 128 * 4 - 1), dict(space=P + 4)):
        assert decode(**kw) == pa.PA_ERR_WORKSPACE, kw
    assert pa.pa_decode_weights_workspace_size(2, 8, 2, 64, 16, 121) == 2 * 8 * 128 * 4
    assert pa.pa_decode_weights_workspace_size(2, 7, 2, 64, 16, 121) == 0

    def prompt(w=P, ws=128, q=P, qdt=1, k=P, kdt=1, bt=P, cl=P, qs=P, B=2, T=50, hq=8, hkv=2, D=64, bs=16, mb=8, nb=20,
               mq=40, mc=128, scale=0.1, decay=1.0, window=0):
        return lib.pa_prefill_weights(w, ws, q, qdt, k, kdt, bt, cl, qs, B, T, hq, hkv, D, bs, mb, nb, mq, mc, scale, decay,
                                      window, P, 1 << 30, None)

    assert prompt(B=0) == prompt(T=0) == prompt(mq=0) == prompt(mc=0) == pa.PA_OK
    for kw in (dict(w=None), dict(q=None), dict(k=None), dict(bt=None), dict(cl=None), dict(qs=None), dict(ws=127), dict(T=-1),
               dict(mq=-1), dict(window=-1), dict(mc=129), dict(scale=INF), dict(decay=-1.0), dict(hq=9), dict(q=P + 4),
               dict(k=P + 8), dict(qs=P + 1), dict(w=P + 1)):
        assert prompt(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(D=80), dict(bs=257, mc=100), dict(qdt=0, kdt=1)):
        assert prompt(**kw) == pa.PA_ERR_UNSUPPORTED, kw

    def evict(kept=P, ks=64, nw=P, ns=64, w=2 * P, ws=128, k=P, v=P, dt=1, bt=P, cl=P, nt=P, kl=P, B=2, hkv=2, D=64, bs=16, mb=8,
              mnb=4, nb=20, mc=128, sinks=4, recent=8):
        return lib.pa_evict(kept, ks, nw, ns, w, ws, k, v, dt, bt, cl, nt, kl, B, hkv, D, bs, mb, mnb, nb, mc, sinks, recent, None)

    assert evict(B=0) == evict(ks=0) == evict(mc=0) == pa.PA_OK
    for kw in (dict(kept=None), dict(nw=None), dict(w=None), dict(k=None), dict(v=None), dict(bt=None), dict(cl=None),
               dict(nt=None), dict(kl=None), dict(ws=127), dict(mc=129), dict(sinks=-1), dict(recent=-1), dict(dt=4),
               dict(mnb=0), dict(nb=0), dict(B=-1), dict(hkv=0), dict(D=0), dict(bs=0), dict(w=P), dict(k=P + 8),
               dict(kept=P + 2), dict(ks=-1)):
        assert evict(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(D=4), dict(B=70000), dict(D=7, dt=0), dict(hkv=65535 * 16 + 1),
               dict(mc=(1 << 30) + 1, mb=1 << 30, ws=1 << 31)):
        assert evict(**kw) == pa.PA_ERR_UNSUPPORTED, kw


def test_binding_refuses_mismatched_tensors():
    B, hq, hkv, D, bs = 2, 4, 2, 64, 16
    k, v, q = torch.zeros(8, bs, hkv, D), torch.zeros(8, bs, hkv, D), torch.zeros(B, hq, D)
    tables, lens = torch.zeros(B, 4, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    w, ws = torch.zeros(B, hkv, 64), torch.zeros(64, dtype=torch.uint8)
    ok = dict(out=q.clone(), weights=w, query=q, k_cache=k, v_cache=v, block_tables=tables, context_lens=lens,
              max_context_len=64, scale=1.0, workspace=ws)
    with pytest.raises(ValueError):    # not on a CUDA device
        pa.pa_decode_weights(**ok)
    for err, kw in ((TypeError, dict(weights=w.double())), (ValueError, dict(weights=w[:, :1])), (ValueError, dict(weights=w[:, :, :63])),
                    (ValueError, dict(out=q[:1])), (TypeError, dict(query=q.half(), out=q.half())), (TypeError, dict(block_tables=tables.long())),
                    (TypeError, dict(context_lens=lens.long())), (ValueError, dict(v_cache=v[:4])), (ValueError, dict(k_cache=k[0]))):
        with pytest.raises(err):
            pa.pa_decode_weights(**dict(ok, **kw))
    ok = dict(weights=w, query=q, k_cache=k, block_tables=tables, context_lens=lens, query_start=torch.zeros(3, dtype=torch.int32),
              max_query_len=1, max_context_len=64, scale=1.0, workspace=ws)
    for err, kw in ((ValueError, {}), (TypeError, dict(query_start=lens)), (TypeError, dict(query=q.half())), (ValueError, dict(query=q[..., :32])),
                    (TypeError, dict(weights=w.half()))):
        with pytest.raises(err):
            pa.pa_prefill_weights(**dict(ok, **kw))
    ok = dict(kept=torch.zeros(B, hkv, 8, dtype=torch.int32), new_weights=w.clone(), weights=w, k_cache=k, v_cache=v, block_tables=tables,
              context_lens=lens, new_tables=tables, keep_lens=lens, max_context_len=64)
    for err, kw in ((ValueError, {}), (TypeError, dict(kept=w)), (TypeError, dict(kept=torch.zeros(B, 1, 8, dtype=torch.int32))),
                    (TypeError, dict(keep_lens=lens.long())), (ValueError, dict(v_cache=v.half())), (TypeError, dict(new_tables=tables[:1])),
                    (ValueError, dict(weights=w[:, :, :8].contiguous()))):
        with pytest.raises(err):
            pa.pa_evict(**dict(ok, **kw))
    x, pos, f = torch.zeros(3, 2, D), torch.zeros(3, dtype=torch.int32), torch.zeros(D // 2, dtype=torch.float64)
    for err, weight in ((ValueError, torch.ones(D)), (TypeError, torch.ones(D - 1)), (TypeError, torch.ones(D).half())):
        with pytest.raises(err):
            pa.pa_norm_rope(x.clone(), x, weight, 1e-6, pos, f)
        with pytest.raises(err):
            pa.pa_norm_rope_backward(x.clone(), torch.zeros(D), x, x, weight, 1e-6, pos, f, ws)
    with pytest.raises(TypeError):
        pa.pa_norm_rope_backward(x.clone(), torch.zeros(D).half(), x, x, torch.ones(D), 1e-6, pos, f, ws)


def test_compact_takes_fresh_blocks_and_releases_the_old_ones():
    bm = pa.BlockManager(12, 16)                   # usable blocks 1 .. 11
    bm.allocate(7, 70)                             # 1 .. 5
    assert bm.compact(7, 33) == [6, 7, 8]
    assert bm.block_table(7) == [6, 7, 8] and bm.num_tokens(7) == 33
    assert bm.free_list() == [1, 2, 3, 4, 5, 9, 10, 11]
    slot, src, dst = bm.append_slot(7)             # goes on in the third block
    assert (slot, src, dst) == (8 * 16 + 1, -1, -1)
    assert bm.compact(7, 0) == [] and bm.num_tokens(7) == 0
    assert bm.append_slot(7)[0] == 6 * 16          # (6 was released to the front)


def test_compact_leaves_a_fork_its_blocks_and_refusals_change_nothing():
    bm = pa.BlockManager(8, 16)                    # 7 usable
    bm.allocate(0, 64)                             # 1 .. 4
    bm.fork(0, 1)
    state = lambda: (bm.block_table(0), bm.block_table(1), bm.free_list(), bm.stats())  # noqa: E731
    before = state()
    for args, status in (((0, 65), pa.PA_ERR_INVALID_ARG), ((0, 64), pa.PA_ERR_OUT_OF_BLOCKS), ((9, 1), pa.PA_ERR_NOT_FOUND),
                         ((0, -1), pa.PA_ERR_INVALID_ARG)):
        with pytest.raises(pa.PAError) as e:
            bm.compact(*args)
        assert e.value.status == status and state() == before
    assert bm.compact(0, 40) == [5, 6, 7]
    assert bm.block_table(1) == [1, 2, 3, 4] and bm.refcount(1) == 1 and bm.free_list() == []
    bm.free(1)
    bm.enable_swap(8)
    bm.swap_out([0])
    with pytest.raises(pa.PAError) as e:
        bm.compact(0, 10)
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    assert np.array_equal(bm.swap_in([0])[:, 0], [0, 1, 2])
