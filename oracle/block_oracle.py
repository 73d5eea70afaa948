"""CPU oracle of the MoE block around the LoRA path -- test infrastructure.

numpy in float64, from the operators' definitions: the norm between blocks, the
router's choice, the experts and the 4-bit rows. It shares no code with the product path;
inputs are float64 arrays of the values the device holds.
"""

from __future__ import annotations

import numpy as np


def rms(v, w, eps):
    return v * w / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)


def block_norm(y, residual, pre, post=None, gate=None, scale=1.0, eps=1e-6):
    """(residual_out, normed or None), unrounded."""
    n = y if post is None else rms(y, post, eps)
    if gate is not None:
        n = n * gate
    r = residual + scale * n
    return r, None if pre is None else rms(r, pre, eps)


def moe_route(logits, topk, renormalize=True, scale=1.0):
    """(ids int32 [T, topk], weights float64 [T, topk]); loops over rows and rounds."""
    T, E = logits.shape
    ids = np.full((T, topk), -1, np.int32)
    weights = np.zeros((T, topk))
    for t in range(T):
        takeable = [e for e in range(E) if logits[t, e] > -np.inf]
        order = sorted(takeable, key=lambda e: (-logits[t, e], e))
        if not order:
            continue
        top = logits[t, order[0]]
        soft = {e: 1.0 if logits[t, e] == top else np.exp(logits[t, e] - top) for e in takeable}
        took = order[:topk]
        total = sum(soft[e] for e in (took if renormalize else takeable))
        for j, e in enumerate(took):
            ids[t, j], weights[t, j] = e, scale * soft[e] / total
    return ids, weights


def w4_values(qweight, scales, K, group):
    """float64 weight rows [N, K] of packed bytes uint8 [N, Kp/2] and scales float64 [N, Kp/group]."""
    N = qweight.shape[0]
    words = np.ascontiguousarray(qweight).view("<u4")
    out = np.zeros((N, K))
    for k in range(K):
        block, i, t, j = k // 128, k % 128 // 32, k % 32 // 8, k % 8
        bit = 4 * (j // 2) + (16 if j % 2 else 0)
        q = (words[:, block * 16 + 4 * t + i] >> np.uint32(bit)) & np.uint32(15)
        out[:, k] = scales[:, k // group] * (q.astype(np.float64) - 8)
    return out


def moe_gate_up(x, ids, w, delta=None):
    """(act [T * topk, I], its condition: sum of magnitudes that bounds an accumulation's error)."""
    T, k = ids.shape
    E, I2, _ = w.shape
    act = np.full((T * k, I2 // 2), np.nan)
    slack = np.zeros_like(act)
    for i in range(T * k):
        e = ids.reshape(-1)[i]
        if not 0 <= e < E:
            continue
        v = w[e] @ x[i // k]
        m = np.abs(w[e]) @ np.abs(x[i // k])
        if delta is not None:
            v, m = v + delta[i], m + np.abs(delta[i])
        g, u = v[:I2 // 2], v[I2 // 2:]
        s = g / (1 + np.exp(-g))
        act[i] = s * u
        slack[i] = 1.1 * m[:I2 // 2] * np.abs(u) + np.abs(s) * m[I2 // 2:]
    return act, slack


def moe_down(act, ids, weights, w, delta=None):
    """(out [T, H], sum of magnitudes behind each value)."""
    T, k = ids.shape
    E, H, _ = w.shape
    out, mag = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e, i = ids[t, j], t * k + j
            if not 0 <= e < E:
                continue
            v, m = w[e] @ act[i], np.abs(w[e]) @ np.abs(act[i])
            if delta is not None:
                v, m = v + delta[i], m + np.abs(delta[i])
            out[t] += weights[t, j] * v
            mag[t] += abs(weights[t, j]) * m
    return out, mag
