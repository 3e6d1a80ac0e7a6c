"""Rotary positions in both pair layouts, a paged key/value cache and attention over it, fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages name rotary embedding and LLM inference (hada.io FA3 summary, "Niedrige FP8-Präzision
und incoherent processing", "Weitere Optimierungen und künftige Integration") and define neither
a cache nor a drafted tree.  Readings:

* rotation: RoFormer's (module ``rope``) on the first ``rot`` elements of a row, pairs (2i, 2i+1) or
  (i, i + rot/2), frequencies optionally stretched by a factor: "linear" theta / f, "ntk" base *
  f^(rot/(rot-2)), "yarn" by parts (Peng et al. 2023): with r turns within the original length and
  g = clamp((r - 1) / 31, 0, 1), theta' = (1 - g) theta / f + g theta, cos and sin times
  0.1 ln f + 1.  The gradient is the transposed matrix.
* cache row, E4M3: scale = max|x| / 448 (1 for a row of zeros), code = E4M3(x / scale).
* attention: drafted token t of sequence b sees the keys before the drafts and drafted key i
  where bit i of mask[b][t] is set (no mask: i <= t); a row that sees nothing gives 0 and -inf.
"""

import numpy as np

from . import e4m3

__all__ = ["frequencies", "rotate", "quantise_rows", "tree_attention"]


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, length=0.0):
    """(theta [rot/2], multiplier of cos and sin)."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    th = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return th / factor, 1.0
    if scaling == "yarn":
        g = np.clip((length * th / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
        return (1 - g) * th / factor + g * th, 0.1 * np.log(factor) + 1.0
    return th, 1.0


def rotate(x, pos, theta, gain=1.0, half=False, transpose=False):
    """x [T, H, D] turned at positions pos [T]; the elements past 2 * len(theta) stay."""
    x = np.asarray(x, dtype=np.float64)
    rot = 2 * len(theta)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * theta[None]
    c, s = gain * np.cos(ang)[:, None], gain * np.sin(ang)[:, None]
    if transpose:
        s = -s
    a_at = np.arange(rot // 2) if half else np.arange(0, rot, 2)
    b_at = a_at + rot // 2 if half else a_at + 1
    out = x.copy()
    out[..., a_at] = x[..., a_at] * c - x[..., b_at] * s
    out[..., b_at] = x[..., a_at] * s + x[..., b_at] * c
    return out


def quantise_rows(x):
    """(codes uint8, scale, pre-rounding quotients) of the rows of x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.abs(x).max(-1)
    scale = np.where(amax > 0, amax / 448.0, 1.0)
    pre = x / scale[..., None]
    return e4m3.encode(pre), scale, pre


def tree_attention(q, k, v, ctx, mask, scale):
    """One sequence: q [T, Hq, D], k, v [ctx + T, Hkv, D], mask [T] ints (or None) ->
    (o [T, Hq, D], lse [Hq, T], spread [T, Hq, D], reach [Hq, T]); spread = sum_j p_j |v_j| and
    reach = max_j scale * sum_d |q_d k_jd| over the seen keys, for error bounds."""
    T, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    o, lse = np.zeros((T, Hq, D)), np.full((Hq, T), -np.inf)
    spread, reach = np.zeros((T, Hq, D)), np.zeros((Hq, T))
    for t in range(T):
        m = (1 << (t + 1)) - 1 if mask is None else int(mask[t]) & 0xFFFFFFFFFFFFFFFF
        seen = np.array([j < ctx or bool((m >> (j - ctx)) & 1) for j in range(L)], dtype=bool)
        if not seen.any():
            continue
        for h in range(Hq):
            kk, vv = k[seen, h * Hkv // Hq], v[seen, h * Hkv // Hq]
            x = scale * (kk @ q[t, h])
            top = x.max()
            p = np.exp(x - top)
            lse[h, t] = top + np.log(p.sum())
            p /= p.sum()
            o[t, h] = p @ vv
            spread[t, h] = p @ np.abs(vv)
            reach[h, t] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return o, lse, spread, reach
