"""Angles far out: positions to the ends of int32 with frequencies up to a thousand radians a
position, where the angle is taken from exact fractions (position and inverse frequency are
rational numbers, 2 pi to 70 digits).  The weight gradient of a single row is in fp32 and holds
the sine and cosine of each pair's angle to within 2^-20 max |dy| |u| (test_qknorm_gpu.py's
docstring: g is off by 2^-21 max |dy|), an angle's 2^-32 of a turn among it."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164, 10 ** 70)


def _angle(position: int, inv_freq: float) -> float:
    turns = position * Fraction(inv_freq) / (2 * PI)
    return float((turns - (turns.numerator // turns.denominator)) * 2 * PI)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,top", [(64, 1.0), (64, 1000.0), (128, 37.0), (128, 1e-4)])
@pytest.mark.parametrize("position", [3, 1 << 20, (1 << 31) - 1, -(1 << 31), -1234567890])
def test_angles_are_as_exact_far_out_as_near(position, d, top, interleaved):
    from padded_variable_length_b200 import binding as Bd
    g = torch.Generator().manual_seed(d)
    x, dy = (torch.randn(1, 1, d, generator=g).to(torch.bfloat16) for _ in range(2))
    inv = top * 10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)
    ang = np.array([_angle(position, float(f)) for f in inv])
    c, s = np.cos(ang), np.sin(ang)
    xs, gs = x[0, 0].double().numpy(), dy[0, 0].double().numpy()
    i, j = (np.arange(0, d, 2), np.arange(1, d, 2)) if interleaved else (np.arange(d // 2), np.arange(d // 2, d))
    ref = gs.copy()
    ref[i], ref[j] = gs[i] * c + gs[j] * s, gs[j] * c - gs[i] * s
    u = xs / np.sqrt(np.mean(xs * xs) + 1e-6)
    dw = Bd.qk_norm_rope_bwd(x.cuda(), None, dy.cuda(), None, torch.ones(d, device="cuda"), inv_freq=inv.cuda(), interleaved=interleaved,
                             positions=torch.tensor([position], dtype=torch.int64).to(torch.int32).cuda())[2]
    err = np.abs(dw.cpu().double().numpy() - ref * u)
    assert np.all(err <= 2.0 ** -20 * np.abs(gs).max() * np.abs(u)), err.max()


def test_frequencies_that_are_no_numbers_do_not_turn():
    from padded_variable_length_b200 import binding as Bd
    x = torch.randn(5, 2, 64).to(torch.bfloat16).cuda()
    inv = torch.full((32,), float("nan"), dtype=torch.float64)
    inv[::2] = float("inf")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    y = Bd.qk_norm_rope(x, None, inv_freq=inv.cuda(), positions=pos)[0]
    assert torch.equal(y, Bd.qk_norm_rope(x)[0])
