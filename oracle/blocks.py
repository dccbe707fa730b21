"""A decode step over selected pages, restated one element at a time (oracle): positions and slots of the new tokens,
rotary positions, key bounds, page selection and attention over the selected pages."""

from __future__ import annotations

import math

import numpy as np

from . import attention as _a


def token_map(qo_indptr, kv_indptr, kv_indices, last_page_len, page_size: int, offsets=None):
    """(positions, slots) of every new token, int64."""
    pos, slots = [], []
    for i in range(len(qo_indptr) - 1):
        pages = kv_indices[kv_indptr[i]:kv_indptr[i + 1]]
        n = int(qo_indptr[i + 1] - qo_indptr[i])
        L = _a.kv_len_of(len(pages), int(last_page_len[i]), page_size)
        for t in range(n):
            P = _a.query_position(L, n, t)
            pos.append(P + (0 if offsets is None else int(offsets[i])))
            slots.append(int(pages[P // page_size]) * page_size + P % page_size)
    return np.array(pos, np.int64), np.array(slots, np.int64)


def turns(positions, steps) -> np.ndarray:
    """Fraction of a turn of every (position, pair), float64: position * step modulo 2^64, in units of 2^-64."""
    return np.array([[(int(P) * int(s)) % 2 ** 64 / 2.0 ** 64 for s in steps] for P in positions]).reshape(len(positions), len(steps))


def rotate(x, angle, interleaved: bool, amplitude: float = 1.0) -> np.ndarray:
    """x [T, heads, D] with the pairs of its first 2 * angle.shape[1] elements turned by angle [T, pairs] (float64)."""
    y = np.array(x, np.float64)
    half = angle.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = amplitude * np.cos(angle[:, None, i]), amplitude * np.sin(angle[:, None, i])
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def page_bounds(K, scale) -> np.ndarray:
    """Codes [Hkv, 2, D] of one page's valid keys K [keys, Hkv, D] (values that float32 holds), scale [Hkv, D] float32."""
    K = np.asarray(K, np.float32)
    out = np.empty((K.shape[1], 2, K.shape[2]), np.int8)
    with np.errstate(all="ignore"):
        for h in range(K.shape[1]):
            for d in range(K.shape[2]):
                v = K[:, h, d]
                lo, hi = np.min(v) / scale[h, d], np.max(v) / scale[h, d]
                bad = np.isnan(v).any()
                out[h, 0, d] = -127 if bad or np.isnan(lo) else int(np.clip(np.floor(lo), -127, 127))
                out[h, 1, d] = 127 if bad or np.isnan(hi) else int(np.clip(np.ceil(hi), -127, 127))
    return out


def query_codes(q, scale) -> np.ndarray:
    """Whole numbers [G, D] of one KV head's query heads q [G, D] (bf16 values), scale [D]: the float32 steps are the
    definition's."""
    with np.errstate(all="ignore"):
        a = np.asarray(q, np.float32) * np.asarray(scale, np.float32)
        a = np.where(np.isfinite(a), a, np.float32(0))
        top = np.abs(a).max()
        if top == 0:
            return np.zeros(a.shape, np.int64)
        return np.rint((a / top) * np.float32(32767 // len(a))).astype(np.int64)


def select(q, codes, scale, pages, num_blocks: int, num_sink: int, num_recent: int) -> list:
    """Blocks of one (token, KV head): q [G, D], codes [pages, 2, D] of the KV head in page-list order, scale [D]."""
    N = pages
    if N <= num_blocks:
        return list(range(N)) + [-1] * (num_blocks - N)
    c = query_codes(q, scale)
    up, down = np.maximum(c, 0).sum(0), np.minimum(c, 0).sum(0)
    body = range(num_sink, N - num_recent)
    score = {b: int(codes[b, 1].astype(np.int64) @ up + codes[b, 0].astype(np.int64) @ down) for b in body}
    best = sorted(body, key=lambda b: (-score[b], b))[:num_blocks - num_sink - num_recent]
    return list(range(num_sink)) + sorted(best) + list(range(N - num_recent, N))


def attend_blocks(q, k_pool, v_pool, blocks, qo_indptr, kv_indptr, kv_indices, last_page_len, page_size: int,
                  sm_scale: float | None = None):
    """Attention of every one-token request over its selected pages: (o, lse), float64 (pools hold values)."""
    T, Hq, D = q.shape
    group = Hq // k_pool.shape[2]
    scale = 1.0 / math.sqrt(D) if sm_scale is None or sm_scale <= 0 else float(sm_scale)
    o, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    for i in range(len(qo_indptr) - 1):
        if qo_indptr[i + 1] == qo_indptr[i]:
            continue
        r = int(qo_indptr[i])
        pages = np.asarray(kv_indices[kv_indptr[i]:kv_indptr[i + 1]], np.int64)
        L = _a.kv_len_of(len(pages), int(last_page_len[i]), page_size)
        for h in range(k_pool.shape[2]):
            keys = [b * page_size + t for b in blocks[r, h] if b >= 0 for t in range(page_size) if b * page_size + t < L]
            j = np.array(keys)
            K, V = (p[pages[j // page_size], j % page_size, h] for p in (k_pool, v_pool))
            for g in range(h * group, (h + 1) * group):
                o[r, g], lse[r, g] = _a.attend(q[r, g], K, V, 0, len(j) - 1, scale)
    return o, lse
