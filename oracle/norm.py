"""Root-mean-square norm and its gradients (oracle), in float64.

  y = h rstd gain,  rstd = 1 / sqrt(mean(h^2) + eps)
  dh = rstd (gain dy - xhat mean(gain dy xhat)) + dtotal,  xhat = h rstd
  dgain = sum over rows of dy xhat
"""
from __future__ import annotations

import numpy as np


def rstd(h, eps):
    return 1.0 / np.sqrt(np.mean(np.square(h), axis=1, keepdims=True) + eps)


def rms_norm(h, gain, eps):
    h = np.asarray(h, np.float64)
    return h * rstd(h, eps) * np.asarray(gain, np.float64)


def rms_norm_backward(dy, h, gain, eps, dtotal=0.0):
    """(dh, dgain)."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    r = rstd(h, eps)
    xhat, g = h * r, dy * np.asarray(gain, np.float64)
    return r * (g - xhat * np.mean(g * xhat, axis=1, keepdims=True)) + dtotal, (dy * xhat).sum(axis=0)
