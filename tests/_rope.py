"""Plain 64-bit forms of the head norm and the rotation and their error bounds.

Bounds (half a bf16 step is 2^-8 of the value, half a float32 step 2^-24):

* a normed value x r w: the sum of head_dim squares passes 8 + 4 additions of
  positive terms (12 half steps), its root halves that; the mean and eps, the
  root and two products add 5: under 2^-20 of the value in all;
* cosine and sine: the turn's fraction beyond the nearest quarter as float32 is off
  by 2^-27 of a half turn, 2^-25.3 rad, the functions by one step and the amplitude's product by half
  a step: under 2^-22 of the amplitude together (exact frequencies and
  positions); the two products and the sum add 3 half steps of |a| + |b|;
* a turned value: (|a| + |b|) amplitude (2^-20 + 2^-22 + 3 2^-24) < 2^-19 of that
  before it is rounded, 2^-8 of the value when it is.
"""
import math
from fractions import Fraction

import torch

EARLY = 2.0 ** -19

# pi to 192 bits by Machin's formula
_ONE = 1 << 224


def _atan_inverse(n):
    total, term, k, sign = 0, _ONE // n, 1, 1
    while term:
        total += sign * (term // k)
        term //= n * n
        k += 2
        sign = -sign
    return total


_TWO_PI = Fraction(8 * (4 * _atan_inverse(5) - _atan_inverse(239)), _ONE)


def angle(position, inv_freq):
    """position x inv_freq modulo 2 pi, exactly but for the last rounding to 64 bits."""
    t = Fraction(int(position)) * Fraction(float(inv_freq))
    return float(t - _TWO_PI * math.floor(t / _TWO_PI))


def turned(x, positions, inv_freq, axis=None, interleaved=False, amplitude=1.0, w=None, eps=1e-6):
    """float64 norm and rotation of x [T, heads, dim] at positions [T, axes], and
    the bound of its float32 form."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    z, bound = y.clone(), y.abs() * 2.0 ** -20
    half = len(inv_freq)
    if half:
        axis = [0] * half if axis is None else axis
        known = {}
        rows = []
        for at in positions.cpu().tolist():
            row = []
            for a, f in zip(axis, inv_freq):
                if (at[a], f) not in known:
                    known[at[a], f] = angle(at[a], f)
                row.append(known[at[a], f])
            rows.append(row)
        t = torch.tensor(rows, dtype=torch.float64, device=x.device)[:, None]
        i = torch.arange(half, device=x.device)
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = y[..., first], y[..., second]
        z[..., first] = amplitude * (a * t.cos() - b * t.sin())
        z[..., second] = amplitude * (b * t.cos() + a * t.sin())
        bound[..., first] = bound[..., second] = (a.abs() + b.abs()) * abs(amplitude) * EARLY
    return z, bound


def close(got, want, early, what, half_step=2.0 ** -8):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    d = (got - want).abs()
    over = torch.where(torch.isnan(want), torch.zeros_like(d), d - (want.abs() * half_step + early))
    assert d.numel() == 0 or over.max().item() <= 0, f"{what}: over by {over.max().item():.3e}"
