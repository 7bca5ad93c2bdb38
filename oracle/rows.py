"""Oracle of the gated linear recurrence and of the row norms: the definitions in
fp64, token after token and row after row, in plain numpy.

TEST INFRASTRUCTURE, as the rest of this package; it shares no code with the CUDA
library.  ``tests/test_oracle_rows.py`` pins every function against closed forms,
explicit products and finite differences.

Recurrence (page "状态空间与线性注意力", selective-scan reference: per-position a, b,
x, optional initial state, all outputs and the final state), per channel:
``h_t = a_t h_{t-1} + u_t`` with ``a = g`` or ``sigmoid(g)``, ``u = x`` or ``(1 - a) x``.
"""
from __future__ import annotations

import numpy as np

from . import _f64


def gates(g, gate: str):
    """(a, 1 - a) in fp64; the logit form without cancellation."""
    g = _f64(g)
    if gate == "value":
        return g, 1.0 - g
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))


def scan_fwd(x, g, h0=None, gate="value", tied=False):
    """x, g [B,T,D]; returns (h [B,T,D], h_last [B,D])."""
    x = _f64(x)
    a, r = gates(g, gate)
    B, T, D = x.shape
    s = np.zeros((B, D)) if h0 is None else _f64(h0).copy()
    h = np.empty((B, T, D))
    for t in range(T):
        s = a[:, t] * s + (r[:, t] * x[:, t] if tied else x[:, t])
        h[:, t] = s
    return h, s


def scan_bwd(g, h, dh, x=None, h0=None, dh_last=None, gate="value", tied=False):
    """Gradients from the stored outputs h; returns (dx, dg, dh0)."""
    h, dh = _f64(h), _f64(dh)
    x = _f64(x) if tied else None
    a, r = gates(g, gate)
    B, T, D = h.shape
    first = np.zeros((B, D)) if h0 is None else _f64(h0)
    c = np.zeros((B, D)) if dh_last is None else _f64(dh_last).copy()
    dx, dg = np.empty((B, T, D)), np.empty((B, T, D))
    for t in range(T - 1, -1, -1):
        G = dh[:, t] + c
        c = a[:, t] * G
        prev = h[:, t - 1] if t > 0 else first
        da = G * (prev - x[:, t]) if tied else G * prev
        dx[:, t] = r[:, t] * G if tied else G
        dg[:, t] = da * a[:, t] * r[:, t] if gate == "logit" else da
    return dx, dg, c


def norm_fwd(x, w=None, b=None, kind="layer", eps=1e-6):
    """x [R,D]; returns (y, mean or None, rstd)."""
    x = _f64(x)
    D = x.shape[1]
    mean = x.sum(1) / D if kind == "layer" else None
    c = x if mean is None else x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).sum(1) / D + eps)
    y = c * rstd[:, None]
    if w is not None:
        y = y * _f64(w)
    if b is not None:
        y = y + _f64(b)
    return y, mean, rstd


def norm_bwd(dy, x, rstd, mean=None, w=None, kind="layer"):
    """Returns (dx, dw, db)."""
    dy, x, rs = _f64(dy), _f64(x), _f64(rstd)[:, None]
    D = x.shape[1]
    xh = (x - _f64(mean)[:, None]) * rs if kind == "layer" else x * rs
    d = dy if w is None else dy * _f64(w)
    dx = d - xh * ((d * xh).sum(1, keepdims=True) / D)
    if kind == "layer":
        dx = dx - d.sum(1, keepdims=True) / D
    return rs * dx, (dy * xh).sum(0), dy.sum(0)
