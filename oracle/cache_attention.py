"""Attention of a few new tokens over a key/value cache — test infrastructure only.

By definition, row by row: token t of sequence b sees cache rows [0, lengths[b]) and,
where the drafted tokens' rows follow, row lengths[b] + u iff bit u of tree[b][t] is set;
query head h reads key/value head h / (Hq / Hkv). Softmax over the scaled scores of those
rows only (no other row is touched); a row that sees nothing gets O = 0, lse = -inf.
All arithmetic float64.
"""
from __future__ import annotations

import numpy as np


def attend(q, k_cache, v_cache, lengths, tree=None, own_drafts: bool = True, scale=None):
    """q [B, T, Hq, D], caches [B, cap, Hkv, D] -> (o [B, T, Hq, D], lse [B, Hq, T])."""
    q = np.asarray(q, np.float64)
    B, T, Hq, D = q.shape
    G = Hq // k_cache.shape[2]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    o = np.zeros((B, T, Hq, D))
    lse = np.full((B, Hq, T), -np.inf)
    for b in range(B):
        n = int(lengths[b])
        for t in range(T):
            seen = list(range(n))
            if own_drafts:
                word = (1 << (t + 1)) - 1 if tree is None else int(tree[b][t])
                seen += [n + u for u in range(T) if (word >> u) & 1]
            if not seen:
                continue
            k, v = (np.asarray(c[b][seen], np.float64) for c in (k_cache, v_cache))
            for h in range(Hq):
                s = scale * (k[:, h // G] @ q[b, t, h])
                m = s.max()
                e = np.exp(s - m)
                o[b, t, h] = e @ v[:, h // G] / e.sum()
                lse[b, h, t] = m + np.log(e.sum())
    return o, lse
