"""Angles at frequencies far above 1: exact to 2e-7 radians for every finite frequency and every position."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import exact_attention_blackwell_gb300 as fa

BITS = 512


def two_pi():
    """2 pi to 512 bits, by Machin's formula in whole numbers."""
    one = 1 << (BITS + 32)

    def arctan(x):  # of 1 / x
        term = total = one // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total

    return Fraction(8 * (4 * arctan(5) - arctan(239)), one)


TWO_PI = two_pi()
FREQUENCIES = [1000.5, 1e4, 12345.678, -1e5, 1e6, 3.3e7, 1e8, 1e10, -1e15, 1e20, 1e30, 3.4028234663852886e38, 2.0**64, 2.0**100,
               0.99, 1e-3]


def angle(f, position):
    """The angle in (-pi, pi], the fraction of a turn taken exactly."""
    turns = Fraction(f) * position / TWO_PI % 1
    return float((turns - 1 if turns > Fraction(1, 2) else turns) * TWO_PI)


def near_whole_turns(f, count, seed):
    """Positions whose angle is some 1e-5 radians: there a sine shows its angle, which bf16 would hide elsewhere."""
    step = np.uint64(int(Fraction(f) / TWO_PI % 1 * 2**64) % 2**64)
    at = np.random.default_rng(seed).integers(-(2**31), 2**31, 1 << 21)
    part = (at.astype(np.uint64) * step).view(np.int64)  # of a turn, in 2^-64, off by 2^-33 turns
    return at[np.argsort(np.abs(part.astype(np.float64)))[:count]].tolist()


def test_the_model_of_angles():
    assert abs(float(TWO_PI) - 2 * math.pi) < 1e-15 and abs(angle(0.5, 3) - 1.5) < 1e-15 and abs(angle(-0.5, 3) + 1.5) < 1e-15
    for f in FREQUENCIES[:3]:
        assert max(abs(angle(float(np.float32(f)), p)) for p in near_whole_turns(float(np.float32(f)), 3, 1)) < 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [False, True])
def test_angles_at_large_frequencies(pairs):
    """Rows (1, 0) in every pair: cosine and sine of the angle, off by the 2e-7 of the angle and half a step of bf16
    (2^-8 of the value); with gradients (1, 0) the cosine and the negative sine."""
    freq = torch.tensor(FREQUENCIES, dtype=torch.float32)
    n = len(FREQUENCIES)
    values = [float(x) for x in freq]
    positions = [0, 1, -1, 2**31 - 1, -(2**31)]
    for i, f in enumerate(values):
        positions += near_whole_turns(f, 6, seed=i)
    want = torch.tensor([[angle(f, p) for f in values] for p in positions], dtype=torch.float64)
    small = want.abs().amin(0)
    assert (small[:14] < 1e-4).all()  # every large frequency has positions that show its angle
    total = len(positions)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if pairs else (slice(0, n), slice(n, 2 * n))
    x = torch.zeros((total, 2, 64), dtype=torch.bfloat16)
    x[..., a] = 1.0
    x = x.cuda()
    at = torch.tensor(positions, dtype=torch.int32, device="cuda")
    q, k = fa.qk_norm_rope(x, x[:, :1], at, freq.cuda(), interleaved=pairs)
    dq, dk, _, _ = fa.qk_norm_rope_bwd(x, x[:, :1], None, None, at, freq.cuda(), interleaved=pairs)
    torch.cuda.synchronize()
    for y, sign in ((q, 1), (k, 1), (dq, -1), (dk, -1)):
        y = y.cpu().double()
        for got, exact in ((y[..., a], torch.cos(want)), (y[..., b], sign * torch.sin(want))):
            exact = exact[:, None].expand_as(got)
            off = (got - exact).abs()
            assert torch.isfinite(got).all() and (off <= 2e-7 + 2.0**-8 * exact.abs()).all(), (
                f"off by {float(off[exact.abs() < 1e-3].max()):.2e} where the value is below 1e-3")
