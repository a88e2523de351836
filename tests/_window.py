"""Plain 64-bit attention under a mask, with the error bounds of ``_attention``
(which depend on the visible keys alone)."""
import math

import torch


def visible(pos, m, window, sinks):
    """[n, m] truth values: the keys that tokens at positions pos see."""
    j = torch.arange(m, device=pos.device)[None]
    p = pos[:, None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def attend_masked(q, k, v, mask, scale):
    """float64 attention of rows q [n, H, D] over k, v [m, Hk, D] where mask
    [n, m] allows; hidden keys and values do not matter, whatever they are.
    Returns out, lse, and the bounds of both."""
    n, H, D = q.shape
    Hk, m = k.shape[1], k.shape[0]
    out = torch.zeros((n, H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    if m == 0 or n == 0:
        return out, lse, bo, bl
    used = mask.any(0)[:, None, None]
    q = q.double()
    k, v = (torch.where(used, x.double(), torch.zeros((), dtype=torch.float64, device=q.device)) for x in (k, v))
    kk, vv = k.repeat_interleave(H // Hk, 1), v.repeat_interleave(H // Hk, 1)
    s = torch.einsum("nhd,mhd->hnm", q, kk) * scale
    size = torch.einsum("nhd,mhd->hnm", q.abs(), kk.abs()) * abs(scale)
    s = s.masked_fill(~mask[None], -math.inf)
    size = size.masked_fill(~mask[None], 0.0)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("hnm,mhd->nhd", p, vv)
    ds = (2 * (D + 4) * 2.0 ** -24) * size.amax(-1)
    mass = torch.einsum("hnm,mhd->nhd", p, vv.abs())
    lse, ds = lse.T, ds.T
    bo = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * (4 * ds[..., None] + 2.0 ** -20)) * mass
    bl = ds + 2.0 ** -20 + 2.0 ** -22 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    return out, lse, bo, bl
