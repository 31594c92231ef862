"""float64 oracle of the gated linear recurrence with a vector state, token by token (numpy).

    h_t = a_t h_{t-1} + m(g_t) x_t,   o_t = h_t,   a_t = e^{g_t},
    m = 1 ("plain"), 1 - a ("complement"), sqrt(1 - a^2) ("norm"; m = 0 has slope 0)

per (b, h, channel): x, g [B,H,L,D], h0, hT [B,H,D]. Shares no code with the library. g = -inf
gives a = 0: that token starts anew.
"""
from __future__ import annotations

import numpy as np


def input_factor(g, kind):
    """(m(g), dm/dg)."""
    g = np.asarray(g, np.float64)
    if kind == "plain":
        return np.ones_like(g), np.zeros_like(g)
    if kind == "complement":
        return -np.expm1(g), -np.exp(g)
    if kind == "norm":
        m = np.sqrt(-np.expm1(2 * g))
        return m, np.where(m > 0, -np.exp(2 * g) / np.where(m > 0, m, 1), 0.0)
    raise ValueError(kind)


def scan_fwd(x, g, h0=None, kind="plain"):
    """(o [B,H,L,D], hT [B,H,D])."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    B, H, L, D = x.shape
    h = np.zeros((B, H, D)) if h0 is None else np.array(h0, np.float64)
    a, (m, _) = np.exp(g), input_factor(g, kind)
    o = np.empty_like(x)
    for t in range(L):
        h = a[:, :, t] * h + m[:, :, t] * x[:, :, t]
        o[:, :, t] = h
    return o, h


def scan_bwd(x, g, h0, dO, dhT=None, kind="plain"):
    """dict dx, dg, dh0: the gradients of sum(dO * o) + sum(dhT * hT), by back-propagation
    through the token loop."""
    x, g, dO = (np.asarray(v, np.float64) for v in (x, g, dO))
    B, H, L, D = x.shape
    o, _ = scan_fwd(x, g, h0, kind)
    first = np.zeros((B, H, 1, D)) if h0 is None else np.asarray(h0, np.float64)[:, :, None]
    prev = np.concatenate([first, o[:, :, :-1]], 2) if L else o
    a, (m, dm) = np.exp(g), input_factor(g, kind)
    dh = np.zeros((B, H, D)) if dhT is None else np.array(dhT, np.float64)
    dx, dg = np.empty_like(x), np.empty_like(x)
    for t in range(L - 1, -1, -1):
        dh = dh + dO[:, :, t]
        dx[:, :, t] = m[:, :, t] * dh
        dg[:, :, t] = dh * (a[:, :, t] * prev[:, :, t] + dm[:, :, t] * x[:, :, t])
        dh = a[:, :, t] * dh
    return {"dx": dx, "dg": dg, "dh0": dh}
