"""fp64 reference of the paged key-value cache: attention of one new token,
append, eviction, and the accumulated attention weight of a prompt's keys.

TEST INFRASTRUCTURE ONLY (see the package docstring). Everything is the plain
definition, one sequence and head at a time, over NumPy arrays:

    slot j of sequence b lies in page table[b][j // page_size] at j % page_size
    s_j = scale q . k_j,  L = ln sum_j e^(s_j),  o = sum_j e^(s_j - L) v_j
    weight of slot j += sum over the query heads of a key head of e^(s_j - L)
"""

from __future__ import annotations

import numpy as np

__all__ = ["tokens", "paged_decode", "cache_append", "evict_places", "cache_evict", "key_weights"]


def tokens(cache, table, b, n):
    """[Hkv, n, d]: the first n slots of sequence b of a [P, Hkv, ps, d] cache."""
    ps = cache.shape[2]
    out = np.zeros((cache.shape[1], n, cache.shape[3]))
    for j in range(n):
        out[:, j] = cache[table[b, j // ps], :, j % ps]
    return out


def paged_decode(q, k_cache, v_cache, table, lens, scale, visible=None):
    """(o [B, Hq, d], lse [B, Hq], p): p[b] is [Hkv, lens[b]], the weights summed
    over each group. ``visible[b]`` (bool [lens[b]]) leaves slots out."""
    B, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    g = Hq // Hkv
    o, lse, ps = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf), []
    for b in range(B):
        n = int(lens[b])
        k, v = tokens(k_cache, table, b, n), tokens(v_cache, table, b, n)
        w = np.zeros((Hkv, n))
        see = np.ones(n, bool) if visible is None else visible[b]
        for x in range(Hq):
            h = x // g
            s = scale * (k[h][see] @ q[b, x])
            if s.size == 0:
                continue
            m = s.max()
            lse[b, x] = m + np.log(np.exp(s - m).sum())
            p = np.exp(s - lse[b, x])
            o[b, x] = p @ v[h][see]
            w[h][see] += p
        ps.append(w)
    return o, lse, ps


def cache_append(new, cache, table, lens, num_new):
    """A copy of the cache with new [B, Hkv, T, d] written behind lens."""
    out = cache.copy()
    ps = cache.shape[2]
    for b in range(new.shape[0]):
        for i in range(int(num_new[b])):
            j = int(lens[b]) + i
            out[table[b, j // ps], :, j % ps] = new[b, :, i]
    return out


def evict_places(weights, n, budget, recent):
    """Which old slot each new slot holds, for one head: weights [>= n], recent
    bool [>= n] (kept first). Sorted by (recent, weight, lower slot)."""
    if n <= budget:
        return list(range(n))

    def rank(j):
        if recent[j]:  # recent tokens are equal among themselves
            return (False, False, 0.0, j)
        w = float(weights[j])
        return (True, w != w, -w if w == w else 0.0, j)

    kept = sorted(sorted(range(n), key=rank)[:budget])
    stay = {j for j in kept if j < budget}
    movers = iter(j for j in kept if j >= budget)
    return [j if j in stay else next(movers) for j in range(budget)]


def cache_evict(k_cache, v_cache, table, lens, weights, budget, recent, positions=None, next_pos=None):
    """(k_cache, v_cache, weights, positions, lens) after the eviction, copies."""
    k, v, w = k_cache.copy(), v_cache.copy(), weights.copy()
    pos = None if positions is None else positions.copy()
    B, Hkv, _ = weights.shape
    ps = k.shape[2]
    left = []
    for b in range(B):
        n = int(lens[b])
        left.append(min(n, budget))
        for h in range(Hkv):
            if positions is None:
                first = np.arange(n) >= n - recent
            else:
                first = positions[b, h, :n] >= int(next_pos[b]) - recent
            if recent == 0:
                first = np.zeros(n, bool)
            for j, i in enumerate(evict_places(weights[b, h], n, budget, first)):
                for dst, src in ((k, k_cache), (v, v_cache)):
                    dst[table[b, j // ps], h, j % ps] = src[table[b, i // ps], h, i % ps]
                w[b, h, j] = weights[b, h, i]
                if pos is not None:
                    pos[b, h, j] = positions[b, h, i]
    return k, v, w, pos, np.array(left, np.int32)


def key_weights(q, k, lse, causal, scale, q_lens=None):
    """[B, Hkv, Nk] column sums of e^(scale q k^T - lse) over the queries that see
    each key and the query heads of each key head."""
    B, Hq, N, _ = q.shape
    Hkv, Nk = k.shape[1:3]
    out = np.zeros((B, Hkv, Nk))
    for b in range(B):
        n = N if q_lens is None else int(q_lens[b])
        for x in range(Hq):
            h = x // (Hq // Hkv)
            p = np.exp(scale * (q[b, x, :n] @ k[b, h].T) - lse[b, x, :n, None])
            if causal:
                p = np.where(np.arange(Nk)[None, :] <= np.arange(n)[:, None], p, 0.0)
            out[b, h] += p.sum(0)
    return out
