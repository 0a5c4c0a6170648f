"""Routing by softmax or sigmoid scores with a selection bias and expert groups
(oracle), in float64, and the gradient of its weights.

Per token: scores s (sigmoid of each logit, or the softmax over all experts),
selection values v = s + bias; the ``top_groups`` groups whose rank (largest
v, or the sum of the two largest) is highest; the k experts of those groups
with the largest v, descending, ties to the lower id; weights scale * s,
divided by their sum over the k if renormalised. A NaN logit counts as -inf,
+inf as the largest finite fp32; renormalised weights whose sum is 0 are 0.
"""
from __future__ import annotations

import numpy as np


def _clean(logits) -> np.ndarray:
    l = np.asarray(logits, dtype=np.float32).astype(np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    return np.minimum(l, float(np.finfo(np.float32).max))


def _sigmoid(l):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-l))


def _softmax(l):
    """Over the last axis; all zero where every entry is -inf."""
    m = l.max(axis=-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(l == -np.inf, 0.0, np.exp(l - m))
    s = e.sum(axis=-1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def scores(logits, score: str) -> np.ndarray:
    l = _clean(logits)
    return _sigmoid(l) if score == "sigmoid" else _softmax(l)


def _descending(v) -> np.ndarray:
    """Order of each row, largest first, equal values in ascending index."""
    return np.argsort(-v, axis=-1, kind="stable")


def weights(logits, topk_idx, score: str, renormalise: bool, scale: float) -> np.ndarray:
    idx = np.asarray(topk_idx, dtype=np.int64)
    if score == "softmax" and renormalise:  # the softmax of the selected logits
        return scale * _softmax(np.take_along_axis(_clean(logits), idx, axis=1))
    s = np.take_along_axis(scores(logits, score), idx, axis=1)
    if renormalise:
        total = s.sum(axis=1, keepdims=True)
        s = s / np.where(total == 0, 1.0, total)
    return scale * s


def route(logits, top_k, bias=None, score="sigmoid", num_groups=1, top_groups=1,
          group_rank="top2", renormalise=True, scale=1.0):
    """(topk_idx [T, k] int32, topk_w [T, k] float64)."""
    T, E = np.shape(logits)
    v = scores(logits, score)
    if bias is not None:
        with np.errstate(invalid="ignore"):
            v = v + np.asarray(bias, dtype=np.float32).astype(np.float64)
        v = np.where(np.isnan(v), -np.inf, v)
    allowed = np.ones((T, E), dtype=bool)
    if top_groups < num_groups:
        size = E // num_groups
        ranked = np.sort(v.reshape(T, num_groups, size), axis=2)[:, :, ::-1]
        with np.errstate(invalid="ignore"):
            rank = ranked[:, :, 0] + ranked[:, :, 1] if group_rank == "top2" and size > 1 \
                else ranked[:, :, 0]
        rank = np.where(np.isnan(rank), -np.inf, rank)
        kept = _descending(rank)[:, :top_groups]
        group_ok = np.zeros((T, num_groups), dtype=bool)
        np.put_along_axis(group_ok, kept, True, axis=1)
        allowed = np.repeat(group_ok, size, axis=1)
    idx = np.empty((T, top_k), dtype=np.int32)
    for t in range(T):
        cand = np.flatnonzero(allowed[t])
        idx[t] = cand[_descending(v[t, cand])[:top_k]]
    return idx, weights(logits, idx, score, renormalise, scale)


def route_backward(logits, topk_idx, grad_w, score="sigmoid", renormalise=True, scale=1.0):
    """grad_logits [T, E] float64: the Jacobian of ``weights`` (the choice held
    fixed) applied to grad_w. Ids outside [0, E) are skipped, repeats summed."""
    l = _clean(logits)
    T, E = l.shape
    idx = np.asarray(topk_idx, dtype=np.int64)
    ok = (idx >= 0) & (idx < E)
    safe = np.where(ok, idx, 0)
    g = np.where(ok, np.asarray(grad_w, dtype=np.float64), 0.0)
    out = np.zeros((T, E))
    rows = np.broadcast_to(np.arange(T)[:, None], idx.shape)
    if score == "sigmoid":
        ls = np.where(ok, np.take_along_axis(l, safe, axis=1), -np.inf)
        p = _sigmoid(ls)
        slope = p * _sigmoid(-ls)
        if renormalise:
            S = p.sum(axis=1, keepdims=True)
            one = np.where(S == 0, 1.0, S)
            g = np.where(S == 0, 0.0, (g - (g * p).sum(axis=1, keepdims=True) / one) / one)
        d = g * slope
    elif renormalise:
        q = _softmax(np.where(ok, np.take_along_axis(l, safe, axis=1), -np.inf))
        d = q * (g - (g * q).sum(axis=1, keepdims=True))
    else:
        p = _softmax(l)
        sel = np.where(ok, np.take_along_axis(p, safe, axis=1), 0.0)
        inner = (g * sel).sum(axis=1, keepdims=True)
        np.add.at(out, (rows[ok], safe[ok]), g[ok])
        return scale * p * (out - inner)
    np.add.at(out, (rows[ok], safe[ok]), d[ok])
    return scale * out
