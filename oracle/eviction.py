"""Accumulated attention weights and eviction by them, restated one key at a time (oracle)."""

from __future__ import annotations

import math

import numpy as np

from . import attention as _a


def key_weights(q, K, lo: int, hi: int, scale: float, group: int) -> np.ndarray:
    """Weights [kv_len, Hkv] of one query row: sum over the query heads of each KV head of softmax over
    keys lo..hi (float64; q [Hq, D], K [kv_len, Hkv, D]); keys outside the range have weight 0."""
    out = np.zeros(K.shape[:2])
    for h in range(q.shape[0]):
        kvh = _a.kv_head_of(h, group)
        s = (K[lo:hi + 1, kvh] @ q[h]) * scale
        e = np.exp(s - s.max())
        out[lo:hi + 1, kvh] += e / e.sum()
    return out


def add_weights(scores, q, k_pool, kv_indptr, kv_indices, last_page_len, qo_indptr, page_size: int, window_left: int = -1,
                sm_scale: float | None = None) -> None:
    """scores [P, Hkv, ps] (float64, in place) += the weights of every request with one new token."""
    Hq, D = q.shape[1:]
    group = Hq // k_pool.shape[2]
    scale = 1.0 / math.sqrt(D) if sm_scale is None or sm_scale <= 0 else float(sm_scale)
    for i in range(len(qo_indptr) - 1):
        if qo_indptr[i + 1] - qo_indptr[i] != 1:
            continue
        pages = np.asarray(kv_indices[kv_indptr[i]:kv_indptr[i + 1]], dtype=np.int64)
        L = _a.kv_len_of(len(pages), int(last_page_len[i]), page_size)
        lo, hi = _a.visible_range(L - 1, window_left)
        w = key_weights(q[qo_indptr[i]], _a.gather_logical(k_pool, pages, L, page_size), lo, hi, scale, group)
        j = np.arange(L)
        scores[pages[j // page_size], :, j % page_size] += w


def kept_positions(scores, budget: int, num_sink: int, num_recent: int) -> list:
    """Old position of the key at each new position, for one unit with the given scores (one per key)."""
    L = len(scores)
    if L <= budget:
        return list(range(L))
    body = list(range(num_sink, L - num_recent))
    rank = sorted(body, key=lambda j: (math.isnan(scores[j]), 0.0 if math.isnan(scores[j]) else -float(scores[j]), j))
    alive = set(rank[:budget - num_sink - num_recent])
    front = budget - num_recent
    movers = [j for j in body if j in alive and j >= front]
    out = []
    for j in range(front):
        out.append(j if j < num_sink or j in alive else movers.pop(0))
    assert not movers
    return out + list(range(L - num_recent, L))


def evict(pools, scores, kv_indptr, kv_indices, last_page_len, page_size: int, budget: int, num_sink: int, num_recent: int):
    """Evict in place.  pools: arrays [P, ps, H, ...] moved together with scores [P, H, ps].
    Returns kept [B, H, budget] int32 (-1 behind a request's end)."""
    B, H = len(kv_indptr) - 1, scores.shape[1]
    kept = np.full((B, H, budget), -1, dtype=np.int32)
    for i in range(B):
        pages = np.asarray(kv_indices[kv_indptr[i]:kv_indptr[i + 1]], dtype=np.int64)
        L = _a.kv_len_of(len(pages), int(last_page_len[i]), page_size)
        for h in range(H):
            j = np.arange(L)
            old = kept_positions(scores[pages[j // page_size], h, j % page_size], budget, num_sink, num_recent) if L else []
            kept[i, h, :len(old)] = old
            src, dst = np.array(old, dtype=np.int64), np.arange(len(old))
            sp, so, dp, do = pages[src // page_size], src % page_size, pages[dst // page_size], dst % page_size
            for pool in pools:
                pool[dp, do, h] = pool[sp, so, h].copy()
            scores[dp, h, do] = scores[sp, h, so].copy()
    return kept
