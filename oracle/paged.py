"""Oracle of the rotary positions, the paged cache and the attention over it, in 64 bits.

TEST INFRASTRUCTURE (see the package docstring for who may call it).

Definitions: the ones beside sp_rotary, sp_cache_kind, sp_batch and sp_attend in include/specprefill.h.
"""
from __future__ import annotations

import numpy as np

LARGEST = {"e4m3": 448.0, "int8": 127.0}


def rotary(x, positions, inv_freq, axis_of_pair, interleaved=False, inverse=False):
    """x [T, heads, d] float64, positions [axes, T] -> rotated copy; the first 2 * len(inv_freq) entries turn."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    pairs = len(inv_freq)
    for i in range(pairs):
        # long double: a position of 2^31 leaves 11 bits below the 53 of the fraction of a turn
        angle = np.asarray(positions[axis_of_pair[i]], dtype=np.longdouble) * np.longdouble(inv_freq[i])
        angle = np.fmod(angle, 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))).astype(np.float64)[:, None]
        if inverse:
            angle = -angle
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        out[..., a] = x[..., a] * np.cos(angle) - x[..., b] * np.sin(angle)
        out[..., b] = x[..., b] * np.cos(angle) + x[..., a] * np.sin(angle)
    return out


def quantise(x, kind):
    """Rows x [..., d] -> (the values their codes stand for before the scale, scale [...])."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1)
    scale = np.empty(top.shape)
    for i in np.ndindex(top.shape):
        if not np.isfinite(top[i]):
            scale[i] = np.nan
        elif top[i] == 0:
            scale[i] = 1.0
        else:
            k = -100
            while top[i] > LARGEST[kind] * 2.0 ** k:
                k += 1
            scale[i] = 2.0 ** k
    with np.errstate(invalid="ignore"):
        y = np.where(np.isnan(scale)[..., None], 0.0, x / scale[..., None])
    if kind == "int8":
        return np.rint(y), scale
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.rint(y / step) * step, scale


def places(cu_new, kv_len):
    """(sequence, token) of each row cu_new[0] .. cu_new[B] - 1; a token may be negative."""
    out = []
    for b in range(len(kv_len)):
        n = int(cu_new[b + 1] - cu_new[b])
        out += [(b, int(kv_len[b]) - n + t) for t in range(n)]
    return out


def attend(q, k, v, scale, window=0):
    """One sequence: q [n, H, d], k and v [H_kv, kv, d] float64.  (out [n, H, d], lse [H, n], top [n, H]: the
    largest |scale * q.k| summand sum, and spread [n, H, d]: sum of weight * |v|, for error bounds)."""
    n, H, d = q.shape
    H_kv, kv, _ = k.shape
    out = np.zeros((n, H, d))
    spread = np.zeros((n, H, d))
    lse = np.full((H, n), -np.inf)
    top = np.zeros((n, H))
    for h in range(H):
        g = h // (H // H_kv)
        for t in range(n):
            p = kv - n + t
            first = max(0, p - window + 1) if window else 0
            if p < first:
                continue
            kk, vv = k[g, first:p + 1], v[g, first:p + 1]
            x = scale * (kk @ q[t, h])
            m = x.max()
            e = np.exp(x - m)
            w = e / e.sum()
            out[t, h] = w @ vv
            spread[t, h] = w @ np.abs(vv)
            lse[h, t] = m + np.log(e.sum())
            top[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, top, spread
