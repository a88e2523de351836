"""Plain 64-bit forms of the attention operators and their error bounds.

Bounds, for bf16 outputs of bf16 factors (half a bf16 step is 2^-8 of the
value, half a float32 step 2^-24):

* a score s = scale q.k is a float32 sum of exact products: it is off by at
  most ds = 2 (D + 4) 2^-24 scale sum |q||k| (D additions, the scale, and the
  e4m3 scale's product, doubled because the tensor core may truncate where a
  float32 addition rounds);
* a weight exp(s - max) is off by exp(ds') - 1 <= 2 ds' with ds' = 2 ds (the
  score's and the maximum's) and by 2^-20 of the base-2 exponential and its
  argument's rounding, and once more by 2^-8 where it is rounded to bf16 for
  the product with V (times the e4m3 scale: within the same rounding);
* numerator and denominator each carry the weights' error, the numerator the
  rounding too: |out - ref| <= 2^-8 |ref| + (2^-8 + 2 (4 ds + 2^-20)) sum_j p_j |v_j|;
* lse is off by ds + 2^-20 + 2^-22 |lse|.
"""
import math

import torch


def attend(q, k, v, seen, scale):
    """float64 attention of rows q [n, H, D] over k, v [m, Hk, D]; row i sees
    keys j < seen[i].  Returns out, lse, and the bounds of both."""
    n, H, D = q.shape
    Hk = k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    kk = k.repeat_interleave(H // Hk, 1)
    vv = v.repeat_interleave(H // Hk, 1)
    m = k.shape[0]
    out = torch.zeros((n, H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    if m == 0 or n == 0:
        return out, lse, bo, bl
    s = torch.einsum("nhd,mhd->hnm", q, kk) * scale
    size = torch.einsum("nhd,mhd->hnm", q.abs(), kk.abs()) * abs(scale)
    hidden = torch.arange(m, device=q.device)[None] >= seen.to(q.device)[:, None]
    s = s.masked_fill(hidden[None], -math.inf)
    size = size.masked_fill(hidden[None], 0.0)
    lse = torch.logsumexp(s, -1)                                   # [H, n]
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("hnm,mhd->nhd", p, vv)
    ds = (2 * (D + 4) * 2.0 ** -24) * size.amax(-1)                # [H, n]
    mass = torch.einsum("hnm,mhd->nhd", p, vv.abs())
    lse, ds = lse.T, ds.T
    bo = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * (4 * ds[..., None] + 2.0 ** -20)) * mass
    bl = ds + 2.0 ** -20 + 2.0 ** -22 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    return out, lse, bo, bl


def quantise(x):
    """e4m3 values and scales of rows x [..., D] (bf16), exactly as the cache
    defines them: the value nearest to x 448 / a, ties to even, in float64
    (x and a are bf16, so a quotient within 2^-40 of a midpoint is one)."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(a)
    y = torch.where(bad | (a == 0), torch.zeros_like(x), x * 448.0 / torch.where(bad | (a == 0), torch.ones_like(a), a))
    step = torch.exp2(torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent.double() - 4.0)
    z = y / step
    # snap quotients that are midpoints up to float64 rounding
    half = torch.round(2 * z) / 2
    z = torch.where((z - half).abs() < 2.0 ** -30, half, z)
    return torch.round(z) * step, (a / 448.0)[..., 0]
