"""Oracle of block_sample: the tokens that temperature, top-k, top-p and min-p
keep, their probabilities, and the integer draw.

Plain Python and float64 numpy written from the definition in
include/mxfp4_moe.h, one row at a time; it shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

ONE = 2 ** 40


def kept_tokens(l: np.ndarray, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(kept token ids in ranking order, weights w, integer masses W) of one
    row; None where no logit is above -infinity."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return None
    rank = sorted(range(len(l)), key=lambda v: (-l[v], v))
    if not temperature > 0:
        w = np.zeros(len(l))
        w[rank[0]] = 1.0
        return rank[:1], w, [ONE if v == rank[0] else 0 for v in range(len(l))]
    temperature = min(max(float(temperature), 1e-36), 1e30)
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(l == top, 1.0, np.exp((l - top) / temperature))
    W = [int(math.floor(x * ONE)) for x in w]
    n = top_k if 0 < top_k < len(l) else len(l)
    rank = rank[:n]
    if top_p < 1:
        bar = max(1, math.ceil(float(top_p) * float(sum(W[v] for v in rank))))
        run = 0
        for n, v in enumerate(rank, 1):
            run += W[v]
            if run >= bar:
                break
        rank = rank[:n]
    if min_p > 0:
        low = int(min(float(min_p), 1.0) * ONE)
        rank = [v for r, v in enumerate(rank) if r == 0 or W[v] >= low]
    return rank, w, W


def sample_row(l, u=None, **filters):
    """(token or None, probabilities float64); token -1 and zeros without mass."""
    k = kept_tokens(np.asarray(l), **filters)
    if k is None:
        return -1, np.zeros(len(l))
    rank, w, W = k
    keep = sorted(rank)
    p = np.zeros(len(l))
    p[keep] = w[keep] / math.fsum(w[v] for v in keep)
    if u is None:
        return None, p
    m = sum(W[v] for v in keep) * int(float(u) * 2 ** 24) // 2 ** 24
    run = 0
    for v in keep:
        run += W[v]
        if run > m:
            return v, p
    raise AssertionError("the draw lies below the total mass")


def block_sample(logits, u=None, temperature=None, top_k=None, top_p=None, min_p=None):
    """logits [S, K, V] -> (token [S, K] or None, probs [S, K, V])."""
    S, K, V = logits.shape
    token = np.zeros((S, K), np.int32)
    probs = np.zeros((S, K, V))
    for s in range(S):
        f = {n: t[s].item() for n, t in (("temperature", temperature), ("top_k", top_k),
                                         ("top_p", top_p), ("min_p", min_p)) if t is not None}
        if f.get("top_p", 1.0) != f.get("top_p", 1.0):
            f["top_p"] = 1.0
        for i in range(K):
            t, probs[s, i] = sample_row(logits[s, i], None if u is None else u[s, i], **f)
            token[s, i] = -1 if t is None else t
    return (None if u is None else token), probs
