"""The attention half of a layer in float64 numpy, from the operators' definitions (include/mol_attn.h)."""

from __future__ import annotations

import numpy as np


def rope(x, positions, inv_freq, interleaved=False, magnitude=1.0):
    """x [T, heads, D] with its positions turned into it."""
    x = np.array(x, np.float64)
    n = len(inv_freq)
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    angle = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    a, b = x[..., first], x[..., second]
    x[..., first] = magnitude * (a * np.cos(angle) - b * np.sin(angle))
    x[..., second] = magnitude * (b * np.cos(angle) + a * np.sin(angle))
    return x


def cache_append(k, v, k_cache, v_cache, slots):
    """The caches [pages, page_size, heads, D] with the tokens' rows in their slots."""
    k_cache, v_cache = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    pages, size = k_cache.shape[:2]
    for t, s in enumerate(slots):
        if 0 <= s < pages * size:
            k_cache[s // size, s % size] = k[t]
            v_cache[s // size, s % size] = v[t]
    return k_cache, v_cache


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts=None, scale=1.0, window=0):
    """(out, spread, reach): out [T, heads, D], NaN for rows of no sequence; spread, the weighted
    magnitudes sum_j w_j |v_j|; reach [T, heads], the largest scale * sum_d |q_d k_d| of a seen token."""
    T, Hq, D = q.shape
    pages, size, Hkv, _ = k_cache.shape
    group = Hq // Hkv
    out = np.full(q.shape, np.nan)
    spread, reach = np.zeros(q.shape), np.zeros((T, Hq))
    starts = np.arange(T + 1) if q_starts is None else q_starts
    for b, kv in enumerate(kv_lens):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            row = starts[b] + i
            at = kv - n + i
            seen = [j for j in range(max(0, at - window + 1) if window else 0, at + 1)
                    if 0 <= page_table[b][j // size] < pages]
            out[row] = 0.0
            if not seen:
                continue
            page = [page_table[b][j // size] for j in seen]
            offset = [j % size for j in seen]
            k, v = k_cache[page, offset], v_cache[page, offset]  # [tokens, Hkv, D]
            for h in range(Hq):
                s = scale * (k[:, h // group] @ q[row, h])
                w = np.exp(s - s.max())
                w /= w.sum()
                out[row, h] = w @ v[:, h // group]
                spread[row, h] = w @ np.abs(v[:, h // group])
                reach[row, h] = scale * (np.abs(k[:, h // group]) @ np.abs(q[row, h])).max()
    return out, spread, reach
