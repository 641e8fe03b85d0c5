"""Angles of the rotary kernels at far positions, against 60-digit arithmetic.

The reduced angle is off by at most 2^-65 of a turn a position (the fixed-point
frequency is rounded to nearest) plus 2^-72 of a turn a position and radian of
inv_freq (the rounded 2 / pi), and by one fp32 rounding; sine and cosine by another
two units of fp32: 2^-22 of their value in all, generously."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import paged_kv_cache_121_gb300 as pa

pytestmark = pytest.mark.gpu

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def reduced(position, f):
    """position * f modulo a turn, in (-pi, pi], exactly enough."""
    t = Decimal(position) * Decimal(float(f)) / (2 * PI)
    return (t - t.to_integral_value()) * 2 * PI


@pytest.mark.parametrize("layout", [pa.PA_ROPE_HALF, pa.PA_ROPE_INTERLEAVED])
def test_angles_that_return_to_a_multiple_of_a_turn(layout):
    """Frequencies whose angle at a far position is almost a whole number of turns: the sine is what is left, and
    shows the frequency's own error times the position."""
    getcontext().prec = 60
    rng = np.random.default_rng(1)
    for position in (2 ** 31 - 1, 2 ** 31 - 12345, 2 ** 30 + 7, 1_500_000_001):
        turns = np.unique(np.exp(rng.uniform(np.log(1e3), np.log(position / 7), 64)).astype(np.int64))
        f = np.array([float(2 * PI * int(n) / position) for n in turns])
        pairs = len(f)
        x = torch.zeros(1, 1, 2 * pairs, device="cuda")
        first = torch.arange(pairs) * (2 if layout == pa.PA_ROPE_INTERLEAVED else 1)
        second = first + (1 if layout == pa.PA_ROPE_INTERLEAVED else pairs)
        x[0, 0, first] = 1.0
        out = torch.empty_like(x)
        pa.pa_rope(out, x, torch.tensor([position], dtype=torch.int32, device="cuda"), torch.from_numpy(f).cuda(),
                   layout=layout)
        got = out[0, 0].double().cpu().numpy()
        for i in range(pairs):
            t = float(reduced(position, f[i]))
            tol = position * 2 * np.pi * (2.0 ** -65 + f[i] * 2.0 ** -72) + 2.0 ** -22 * abs(np.sin(t))
            assert abs(got[second[i]] - np.sin(t)) <= tol, (position, f[i])
            assert abs(got[first[i]] - np.cos(t)) <= 2.0 ** -22, (position, f[i])
