"""fp64 reference (NumPy, CPU) of the operators around a paged key-value cache: norm + rotary
position of queries and keys with its gradients, rows rounded to e4m3 with one power of two each,
and attention of the newest rows over keys and values given per sequence.

Imports nothing from the package, so the CUDA path and this reference share no code. The routed
attention and the gate themselves are moba_ref's rules, stated again here for cached sequences.
"""
from __future__ import annotations

import math

import numpy as np


def f64(t) -> np.ndarray:
    """A torch tensor or array in fp64 on the CPU."""
    return t.detach().double().cpu().numpy() if hasattr(t, "detach") else np.asarray(t, np.float64)


# ------------------------------------------------------------------------------ norm + rotary
def pair_index(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(z, rope, pos, interleaved, sign=1.0):
    """Pairs of the first rot elements of z [T, H, d] turned by sign * the angle of pos[t]."""
    rot = rope.shape[1]
    a, b = pair_index(rot, interleaved)
    c = rope[pos][:, None, :rot // 2]
    s = sign * rope[pos][:, None, rot // 2:]
    out = z.copy()
    out[..., a] = z[..., a] * c - z[..., b] * s
    out[..., b] = z[..., b] * c + z[..., a] * s
    return out


def norm_rope(x, w, rope, pos, eps, interleaved):
    """y [T, H, d] of x [T, H, d]."""
    x, w, rope = f64(x), f64(w), f64(rope)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * w, rope, np.asarray(pos), interleaved)


def norm_rope_bwd(x, w, rope, pos, dy, eps, interleaved):
    """(dx, dw, size): the gradients and, for tolerances, the size of the terms that dx sums
    (|dz w| + |x r| |mean|) r, row by row."""
    x, w, rope, dy = f64(x), f64(w), f64(rope), f64(dy)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    hat = x * r
    dz = rotate(dy, rope, np.asarray(pos), interleaved, -1.0)
    dw = (dz * hat).sum((0, 1))
    dh = dz * w
    mean = (dh * hat).mean(-1, keepdims=True)
    dx = r * (dh - hat * mean)
    size = r * (np.abs(dh).max(-1, keepdims=True) + np.abs(hat).max(-1, keepdims=True)
                * np.abs(dh * hat).mean(-1, keepdims=True))
    return dx, dw, size


# ------------------------------------------------------------------------------------- e4m3
def e4m3_values() -> np.ndarray:
    """The 127 finite non-negative values, ascending: code c stands for values[c]."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def quantise(x):
    """(code bytes, scale bytes) of rows x [..., d]: the smallest 2^(b-127) >= 2^-126 that keeps
    the largest magnitude within 448; codes to nearest, ties to the even code."""
    x = f64(x)
    top = np.abs(x).max(-1)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(top / 448.0))
    # log2 may be off by a rounding at the border: settle it on the exact inequality
    e = np.where(top > 0, e, -126.0)
    e = np.where(top / np.exp2(e - 1) <= 448.0, e - 1, e)
    e = np.where(top / np.exp2(e) > 448.0, e + 1, e)
    e = np.maximum(e, -126.0)
    v = e4m3_values()
    y = np.abs(x) / np.exp2(e)[..., None]
    hi = np.clip(np.searchsorted(v, y), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - v[lo], v[hi] - y
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8), (e + 127).astype(np.uint8)


def dequantise(codes, scale):
    v = e4m3_values()
    mag = v[np.minimum(codes & 127, 126)]
    return np.where(codes & 128, -mag, mag) * np.exp2(scale.astype(np.float64) - 127)[..., None]


# ------------------------------------------------------------------------------- attention
def route(q, sums, pos, block, topk):
    """Blocks (ascending) that a row at position pos selects: q [d], sums [blocks, d]."""
    cur = pos // block
    if topk - 1 >= cur:
        return list(range(cur + 1))
    score = sums[:cur] @ q
    order = sorted(range(cur), key=lambda j: (-score[j], j))
    return sorted(order[:topk - 1]) + [cur]


def attend(q, k, v, scale, keys):
    """One row over the listed keys: (o, lse, spread, dot) with spread = sum p |v| and dot the
    largest sum_i |q_i k_i| * scale, which bound the roundings."""
    if len(keys) == 0:
        return np.zeros(v.shape[-1]), -math.inf, np.zeros(v.shape[-1]), 0.0
    kk, vv = k[keys], v[keys]
    z = kk @ q * scale
    m = z.max()
    p = np.exp(z - m)
    return (p @ vv / p.sum(), m + math.log(p.sum()), p @ np.abs(vv) / p.sum(),
            float((np.abs(kk) @ np.abs(q)).max() * scale))


def cached_attention(q, k, v, lens, rows, scale, sums=None, block=None, topk=0):
    """q [nseq * rows, Hq, d]; k, v: per sequence [L_s, Hkv, d]; sums: per sequence [blocks, Hkv,
    d] (topk > 0). Returns o, lse [Hq, n], idx (or None), spread, dot."""
    q = f64(q)
    n, hq, d = q.shape
    o, spread = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, dot = np.full((hq, n), -math.inf), np.zeros((hq, n))
    idx = np.full((hq, n, topk), -1, np.int32) if topk else None
    for s, L in enumerate(lens):
        group = hq // k[s].shape[1]
        for r in range(rows):
            pos = L - rows + r
            if pos < 0:
                continue
            for h in range(hq):
                g, at = h // group, s * rows + r
                keys = np.arange(pos + 1)
                if topk:
                    pick = route(q[at, h], sums[s][:, g], pos, block, topk)
                    idx[h, at, :len(pick)] = pick
                    keys = keys[np.isin(keys // block, pick)]
                o[at, h], lse[h, at], spread[at, h], dot[h, at] = attend(
                    q[at, h], k[s][:, g], v[s][:, g], scale, keys)
    return o, lse, idx, spread, dot
