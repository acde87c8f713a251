"""Oracle of trees of drafted tokens, of the attention weight that cached tokens gather, and of cutting a cache, in 64 bits.

TEST INFRASTRUCTURE (see the package docstring for who may call it).

Definitions: the ones beside sp_tree_seen, sp_attend_tree, sp_tree_accept, sp_attend_weights, sp_cache_choose and
sp_cache_keep in include/specprefill.h.
"""
from __future__ import annotations

import numpy as np


def tree_seen(parent):
    """One sequence: parents [n] -> (seen [n, n] bool, depth [n])."""
    n = len(parent)
    seen, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int64)
    for t in range(n):
        u = t
        while 0 <= u:
            seen[t, u] = True
            up = int(parent[u])
            u = up if 0 <= up < u else -1
        depth[t] = seen[t].sum() - 1
    return seen, depth


def words(seen, count):
    """Rows of truth values [n, m] as uint32 words [n, count]."""
    out = np.zeros((seen.shape[0], count), dtype=np.uint32)
    for t, u in zip(*np.nonzero(seen)):
        out[t, u // 32] |= np.uint32(1) << np.uint32(u % 32)
    return out


def visible(n, kv, window=0, seen=None):
    """[n, kv]: which cached tokens each new token sees; causal, or by the bits of drafted tokens [n, n]."""
    i = np.arange(kv)
    out = np.zeros((n, kv), dtype=bool)
    ctx = kv - n
    for t in range(n):
        p = ctx + t if seen is None else ctx + max(int(seen[t].sum()), 1) - 1
        inside = i > p - window if window else np.ones(kv, dtype=bool)
        if seen is None:
            out[t] = (i <= p) & inside
        else:
            out[t] = (i < ctx) & inside
            for u in range(max(0, -ctx), n):
                out[t, ctx + u] = seen[t, u]
    return out


def attend(q, k, v, scale, see):
    """One sequence: q [n, H, d], k and v [H_kv, kv, d], see [n, kv].  As oracle.paged.attend: (out, lse, top, spread)."""
    n, H, d = q.shape
    group = H // k.shape[0]
    out, spread = np.zeros((n, H, d)), np.zeros((n, H, d))
    lse, top = np.full((H, n), -np.inf), np.zeros((n, H))
    for h in range(H):
        for t in range(n):
            kk, vv = k[h // group][see[t]], v[h // group][see[t]]
            if not len(kk):
                continue
            x = scale * (kk @ q[t, h])
            m = x.max()
            e = np.exp(x - m)
            w = e / e.sum()
            out[t, h], spread[t, h] = w @ vv, w @ np.abs(vv)
            lse[h, t] = m + np.log(e.sum())
            top[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, top, spread


def weights(q, k, lse, scale, see):
    """One sequence: the sum of the weights that q [n, H, d] gives k [H_kv, kv, d] with normalisers lse [H, n]:
    ([H_kv, kv], and a bound on how far fp32 sums of fp32 weights may be from it).

    A logit is off by 2^-24 of the sum of its products' magnitudes for each of its d products and additions, and of itself
    for the factor's roundings; the normaliser and the exponential's argument by 2^-24 of theirs, twice; the exponential by 2^-22
    and its subnormal results are 0; the sum of n terms by n * 2^-24 of it."""
    n, H, d = q.shape
    H_kv, kv, _ = k.shape
    group = H // H_kv
    got, bound = np.zeros((H_kv, kv)), np.zeros((H_kv, kv))
    for h in range(H):
        g = h // group
        for t in range(n):
            if lse[h, t] == -np.inf:
                continue
            kk = k[g][see[t]]
            with np.errstate(invalid="ignore", over="ignore"):
                w = np.exp(scale * (kk @ q[t, h]) - lse[h, t])
                dx = (d + 8) * 2.0 ** -24 * scale * (np.abs(kk) @ np.abs(q[t, h])) + 2.0 ** -22 * abs(lse[h, t]) + 2.0 ** -21
                got[g, see[t]] += w
                bound[g, see[t]] += w * (np.expm1(dx) + n * group * 2.0 ** -24) + 2.0 ** -126
    return got, bound


def choose(w, budget, first, last):
    """The kept tokens of one list by its weights [kv] (fp32 values), ascending."""
    kv = len(w)
    n = min(kv, budget)
    score = np.where(np.isnan(w), -np.inf, w.astype(np.float64) + 0.0)
    nan = np.isnan(w)
    must = [i for i in range(kv) if i < first or i >= kv - last] if n < kv else list(range(kv))
    rest = [i for i in range(kv) if i not in set(must)]
    rest.sort(key=lambda i: (nan[i], -score[i], i))
    return np.array(sorted(must + rest[:n - len(must)]), dtype=np.int64)


def accept(parent, draft, target):
    """One sequence: (accepted new tokens, the target's choice after the last)."""
    n = len(parent)
    if n == 0:
        return [], -1
    path = [0]
    while True:
        cur = path[-1]
        more = [c for c in range(cur + 1, n) if parent[c] == cur and draft[c] == target[cur]]
        if not more:
            return path, int(target[cur])
        path.append(more[0])
