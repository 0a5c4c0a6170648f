"""Dense product with bias, activation and residual, and its gradients
(oracle), in float64.

  z = x w^T + bias,  y = act(z) + residual          x [M, K], w [N, K]
  dz = dy act'(z),   dx = dz w,  dw = dz^T x,  dbias = sum of dz over the rows

act: none, relu, silu z / (1 + e^-z), gelu z Phi(z).
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _phi(z):
    """The normal distribution function."""
    return 0.5 * _erfc(-np.asarray(z, np.float64) / math.sqrt(2.0)) if np.size(z) else np.zeros_like(z)


def act(z, name: str):
    if name == "relu":
        return np.where(z > 0, z, np.where(np.isnan(z), z, 0.0))
    if name == "silu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return z * _phi(z)
    return z


def act_slope(z, name: str):
    z = np.clip(z, -1e4, 1e4)  # the slopes are 0 and 1 there: an infinite z has its limit
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def linear(x, w, bias=None, name="none", residual=None):
    """(y, z)."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = act(z, name)
    return (y if residual is None else y + np.asarray(residual, np.float64)), z


def linear_backward(dy, x, w, name="none", pre=None):
    """(dx, dw, dbias, dz)."""
    dz = np.asarray(dy, np.float64)
    if name != "none":
        dz = dz * act_slope(np.asarray(pre, np.float64), name)
    return dz @ np.asarray(w, np.float64), dz.T @ np.asarray(x, np.float64), dz.sum(axis=0), dz
