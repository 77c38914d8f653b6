"""Oracle of eviction by accumulated attention weight (numpy, fp64).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

weights[row of the sequence][g][j] is the sum, over the decode steps so far and the query heads
of KV head g, of token j's softmax weight.  A context of more than keep tokens keeps its first,
its last and the heaviest of those between, ties to the lower position.
"""
from __future__ import annotations

import numpy as np


def decode_weights(q, k, v, block_tables, context_lens, scale: float):
    """(out [B, H, d], [weights [Hkv, n_i] of this step]) in fp64; q [B, H, d], k / v
    [N, bs, Hkv, d] fp64.  An entry outside the pool stands for rows of zeros."""
    N, bs, Hkv, _ = k.shape
    B, H, d = q.shape
    G = H // Hkv
    out, weights = np.zeros((B, H, d)), []
    for i in range(B):
        n = int(context_lens[i])
        pos = np.arange(n)
        blk = np.asarray(block_tables[i], np.int64)[pos // bs]
        ok = ((blk >= 0) & (blk < N))[:, None, None]
        blk = np.clip(blk, 0, N - 1)
        kk, vv = (np.where(ok, x[blk, pos % bs], 0.0) for x in (k, v))
        w = np.zeros((Hkv, n))
        for h in range(H if n else 0):
            s = (kk[:, h // G] @ q[i, h]) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vv[:, h // G]
            w[h // G] += p
        weights.append(w)
    return out, weights


def select_tokens(weights, rows, context_lens, keep: int, first: int, last: int, new_weights=None):
    """(kept [B, Hkv, keep], kept_lens [B]) int32; new_weights is updated in place."""
    R, Hkv, W = weights.shape
    B = len(rows)
    kept = np.full((B, Hkv, keep), -1, np.int32)
    lens = np.zeros(B, np.int32)
    weights = weights.copy()
    for i in range(B):
        if not 0 <= rows[i] < R:
            continue
        n = max(0, min(int(context_lens[i]), W))
        lens[i] = min(n, keep)
        for g in range(Hkv):
            w = weights[rows[i], g, :n]
            if n <= keep:
                pick = np.arange(n)
            else:
                mid = np.arange(first, n - last)
                key = np.where(np.isnan(w[mid]), -np.inf, w[mid].astype(np.float64))
                # NaN below -inf
                order = np.lexsort((mid, -key, np.isnan(w[mid])))
                pick = np.sort(np.concatenate([np.arange(first), mid[order[: keep - first - last]],
                                               np.arange(n - last, n)]))
            kept[i, g, : len(pick)] = pick
            if new_weights is not None:
                new_weights[rows[i], g] = 0
                new_weights[rows[i], g, : len(pick)] = w[pick]
    return kept, lens


def compact_tokens(cache, kept, kept_lens, block_tables, new_tables) -> None:
    """One tensor [N, bs, Hkv, ...], in place: rows as they were before go to their new places."""
    N, bs = cache.shape[:2]
    was = cache.copy()
    for i in range(kept.shape[0]):
        for g in range(kept.shape[1]):
            r = np.arange(int(kept_lens[i]))
            p = kept[i, g, : len(r)].astype(np.int64)
            src = np.asarray(block_tables[i], np.int64)[p // bs]
            dst = np.asarray(new_tables[i], np.int64)[r // bs]
            cache[dst, r % bs, g] = was[src, p % bs, g]
