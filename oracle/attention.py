"""Oracle of the block's attention: head norms, rotation and append to a paged
cache, and attention over that cache.

Plain float64 numpy written from the definitions of include/mxfp4_moe.h; it
shares no code with the CUDA path.  Arrays hold values (float64), not bf16
bit patterns; nothing is rounded.
"""
from __future__ import annotations

import numpy as np


def head_norm(x: np.ndarray, w, eps: float) -> np.ndarray:
    """x [..., D] -> x / sqrt(mean x^2 + eps) * w (w None: ones)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * w


def rotate(x: np.ndarray, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """Turn the first rot dims of x [..., D] by the angles whose cosines and
    sines the row cos_sin [rot] lists (cosines first)."""
    rot = cos_sin.shape[-1]
    c, s = cos_sin[: rot // 2], cos_sin[rot // 2:]
    y = x.copy()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        y[..., a] = x[..., a] * c[j] - x[..., b] * s[j]
        y[..., b] = x[..., a] * s[j] + x[..., b] * c[j]
    return y


def kv_append(qkv, kv_len, block_table, k_cache, v_cache, q_out, cos_sin=None, q_weight=None,
              k_weight=None, norm=True, eps=1e-6, interleaved=False):
    """Updates k_cache, v_cache and q_out in place.  Returns True iff a token
    was left out for a bad index (page id, table row or cos_sin row)."""
    S, N, heads, D = qkv.shape
    pages, Hkv, page_size, _ = k_cache.shape
    Hq = heads - 2 * Hkv
    bad = False
    for s in range(S):
        for i in range(N):
            pos = max(int(kv_len[s]), 0) - N + i
            if pos < 0:
                continue
            lp, at = divmod(pos, page_size)
            page = int(block_table[s, lp]) if lp < block_table.shape[1] else -1
            if not 0 <= page < pages or (cos_sin is not None and pos >= len(cos_sin)):
                bad = True
                continue
            q, k = qkv[s, i, :Hq], qkv[s, i, Hq:Hq + Hkv]
            if norm:
                q, k = head_norm(q, q_weight, eps), head_norm(k, k_weight, eps)
            if cos_sin is not None:
                q, k = rotate(q, cos_sin[pos], interleaved), rotate(k, cos_sin[pos], interleaved)
            q_out[s, i] = q
            k_cache[page, :, at] = k
            v_cache[page, :, at] = qkv[s, i, Hq + Hkv:]
    return bad


def attention(q, k_cache, v_cache, block_table, kv_len, scale=None, window=0):
    """(out, spread, bad): out [S, N, Hq, D]; spread[s, i, h, d] = the softmax-
    weighted mean of |v_d| over the keys seen (what rounding errors of the
    weights scale with); bad: a seen key's page id, or a kv_len, is out of range
    (such keys are left out, such a slot counts as empty)."""
    S, N, Hq, D = q.shape
    pages, Hkv, page_size, _ = k_cache.shape
    scale = D ** -0.5 if scale is None else scale
    out, spread, bad = np.zeros(q.shape), np.zeros(q.shape), False
    for s in range(S):
        n = int(kv_len[s])
        if n > block_table.shape[1] * page_size:
            bad, n = True, 0
        for i in range(N):
            pos = n - N + i
            j = np.arange(max(0, pos - window + 1) if window else 0, pos + 1)
            page = block_table[s, j // page_size].astype(np.int64)
            ok = (page >= 0) & (page < pages)
            bad = bad or not ok.all()
            j, page = j[ok], page[ok]
            if len(j) == 0:
                continue
            k, v = k_cache[page, :, j % page_size], v_cache[page, :, j % page_size]   # [n, Hkv, D]
            for h in range(Hq):
                g = h // (Hq // Hkv)
                z = k[:, g] @ q[s, i, h] * scale
                p = np.exp(z - z.max())
                p /= p.sum()
                out[s, i, h] = p @ v[:, g]
                spread[s, i, h] = p @ np.abs(v[:, g])
    return out, spread, bad
