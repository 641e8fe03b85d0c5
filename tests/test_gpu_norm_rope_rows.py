"""The norm kernels where there are many rows: two or three of a lane group, whole heads and parts, each type and
layout, against 64 bits (test_gpu_norm_rope.py derives the tolerances). The kernels choose by rows and lane groups: 32
and 31 heads fill two rows of a lane group better than three, 48 and 11 three."""
import pytest
import torch

import paged_kv_cache_121_gb300 as pa
from test_gpu_norm_rope import DT, EPS, backward, case, check_forward, check_grads, forward64, grads64

pytestmark = pytest.mark.gpu

SHAPES = [(257, 32, 128, 128), (641, 31, 64, 64), (257, 48, 128, 128), (1021, 11, 128, 64), (4097, 1, 256, 256), (9001, 3, 64, 64)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_many_rows(dt, interleaved, shape):
    T, H, D, rot = shape
    x, w, pos, f, angle = case(shape, DT[dt], 41)
    xd, wd, pd, fd = x.cuda(), w.cuda(), pos.cuda(), f.cuda()
    out = torch.full((T, H, D), float("nan"), dtype=DT[dt], device="cuda")
    pa.pa_norm_rope(out, xd, wd, EPS, pd, fd, layout=int(interleaved), factor=1.25)
    want, size = forward64(x, w, angle, interleaved, 1.25)
    check_forward(out, want, size, D, 1.25)
    go = torch.randn(T, H, D, generator=torch.Generator().manual_seed(42)).to(DT[dt])
    gx, gw = backward(go.cuda(), xd, wd, pd, fd, interleaved, 1.25)
    check_grads(gx, gw, grads64(x, w, go, angle, interleaved, 1.25))
