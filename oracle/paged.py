"""Token streams over a paged cache, float64: attention of the newest tokens,
the weight each cached token received, and eviction by it.

The pages cache whole frames in order ("Amazon and Reactor tune Trainium for
real-time video generation", section "Three problems for generic compilers");
the paged form per token is this library's own, so its definitions are the ones
stated at the calls in rkv.h, written out here one stream and one head at a
time, in the order of the stream's tokens (no pages: a page table only says
where a token lies).
"""

import numpy as np


def token_visible(L, Lq, window, sinks):
    """bool [Lq, L]: query i is token L - Lq + i and sees token j <= its own
    that is within the last ``window`` (0 = any) or among the first ``sinks``."""
    c = L - Lq + np.arange(Lq, dtype=np.int64)[:, None]
    j = np.arange(L, dtype=np.int64)[None, :]
    seen = j <= c
    if window > 0:
        seen &= (j > c - window) | (j < sinks)
    return seen


def decode_ref(q, k, v, scale, window=0, sinks=0):
    """One stream: q [Lq, Hq, D], k/v [L, H, D] float64.  Returns (o [Lq, Hq,
    D], p [Lq, Hq, L]): a query that sees no token gets zeros."""
    Lq, Hq, D = q.shape
    L, H = k.shape[0], k.shape[1]
    G = Hq // H
    seen = token_visible(L, Lq, window, sinks)
    o, p = np.zeros((Lq, Hq, D)), np.zeros((Lq, Hq, L))
    for h in range(Hq):
        for i in range(Lq):
            idx = np.nonzero(seen[i])[0]
            if idx.size == 0:
                continue
            s = (k[idx, h // G] @ q[i, h]) * scale
            e = np.exp(s - s.max())
            p[i, h, idx] = e / e.sum()
            o[i, h] = p[i, h, idx] @ v[idx, h // G]
    return o, p


def received_weight(p, H):
    """[H, L]: the weight each token of a stream received, per key head, from
    p [Lq, Hq, L]."""
    Lq, Hq, L = p.shape
    return p.reshape(Lq, H, Hq // H, L).sum(axis=(0, 2))


def evict_moves(weight, pos, next_pos, budget, sinks, recent):
    """One stream and key head of L tokens: the moves (source, destination) of
    its eviction to ``budget`` tokens, in order."""
    L = len(weight)
    if L <= budget:
        return []

    def rank(j):
        if pos[j] < sinks or pos[j] >= next_pos - recent:
            return (0, 0.0, j)
        w = float(weight[j])
        return (2, 0.0, j) if np.isnan(w) else (1, -w, j)

    kept = set(sorted(range(L), key=rank)[:budget])
    holes = [j for j in range(budget) if j not in kept]
    moved = [j for j in range(budget, L) if j in kept]
    assert len(holes) == len(moved)
    return list(zip(moved, holes))
