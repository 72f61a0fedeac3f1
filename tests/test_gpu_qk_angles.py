"""Angles of far positions: the cosine and sine of position * inv_freq, with inv_freq a
32-bit number and the angle formed without a rounding (as a fraction), to 6 units of 2^-24
and the result's own half step: a quarter turn's half step in 32 bits is 1.6 units of
angle, cosine and sine add up to 2 of theirs, the turn in 64 bits nothing."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import DEV, F32, UNIT, f64

pytestmark = pytest.mark.gpu
TWO_PI = Fraction(62831853071795864769252867665590057683943387987502116419498891846, 10 ** 64)


def exact(positions, freqs):
    """cos, sin [tokens, pairs]."""
    c, s = np.empty((len(positions), len(freqs))), np.empty((len(positions), len(freqs)))
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            turn = Fraction(p) * Fraction(f) / TWO_PI
            w = float((turn - round(turn)) * TWO_PI)
            c[i, j], s[i, j] = math.cos(w), math.sin(w)
    return c, s


@pytest.mark.parametrize("top", [1e-3, 1.0, 100.0])
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles(interleaved, top):
    D, T = 64, 12
    g = torch.Generator().manual_seed(int(top))
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 0, 1, -1] + torch.randint(
        2 ** 29, 2 ** 31 - 1, (T - 6,), generator=g).tolist()
    f = (top * (0.5 + 0.5 * torch.rand(D // 2, generator=g))).float()
    c, s = exact(pos, f.tolist())
    first = torch.zeros(D)
    first[0::2 if interleaved else 1][:D // 2] = 1.0        # the pairs' first members
    x = first.repeat(1, T, 1).to(DEV)
    k = dict(inv_freq=f.to(DEV), norm="none", interleaved=interleaved,
             positions=torch.tensor([pos], dtype=torch.int32, device=DEV))
    y = f64(osdn.qk_rotary_forward(x, None, D, **k)[0])[0, 0]
    d = f64(osdn.qk_rotary_backward(x, None, x[:, None].contiguous(), None, D, **k)["q"])[0]
    torch.cuda.synchronize()
    a, b = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, D // 2),
                                                                 slice(D // 2, D))
    for got, want in ((y[:, a], c), (y[:, b], s), (d[:, a], c), (d[:, b], -s)):
        worst = np.max(np.abs(got - want) / (6 * UNIT + UNIT * np.abs(want)))
        print("worst error %.3f of its bound" % worst, flush=True)
        assert worst <= 1.0
