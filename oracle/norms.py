"""float64 oracle of the norms before and after a block (numpy). Shares no code with the library.

    addnorm   r = res + alpha rscale x,  y = norm(r) w              (rows [N, D])
    headnorm  y = norm(o) w act(z)                                  (o [B,H,L,D]; z, y [B,L,H,D])
    norm: "rms"    r / sqrt(mean(r^2) + eps)
          "layer"  (r - mean(r)) / sqrt(var(r) + eps)
    act:  "silu"   z / (1 + e^-z),  "sigmoid"  1 / (1 + e^-z),  none without z

The gradients are the norms' Jacobians written out as matrices, row by row: with N = D channels,
C = I - 1 1^T / N for the layer norm (I for the RMS norm) and u = C r,
    d norm / d r = (I / s - u u^T / (N s^3)) C,   s = sqrt(|u|^2 / N + eps).
"""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, np.float64) for x in xs]


def norm(r, kind, eps):
    (r,) = _f64(r)
    u = r - r.mean(-1, keepdims=True) if kind == "layer" else r
    return u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)


def norm_vjp(r, d, kind, eps):
    """d^T (d norm / d r) for every row of r, by the Jacobian matrix."""
    r, d = _f64(r, d)
    D = r.shape[-1]
    C = np.eye(D) - (1.0 / D if kind == "layer" else 0.0)
    out = np.empty(r.shape)
    rr, dd, oo = r.reshape(-1, D), d.reshape(-1, D), out.reshape(-1, D)
    for i in range(rr.shape[0]):
        u = C @ rr[i]
        s = np.sqrt(u @ u / D + eps)
        oo[i] = (dd[i] / s - (dd[i] @ u) * u / (D * s ** 3)) @ C
    return out


def addnorm_fwd(x, res, rscale, w, alpha, kind, eps):
    x, res, rscale, w = _f64(x, res, rscale, w)
    r = alpha * x * (1.0 if rscale is None else rscale) + (0.0 if res is None else res)
    return r, norm(r, kind, eps) * (1.0 if w is None else w)


def addnorm_bwd(x, r, rscale, w, dy, dr, alpha, kind, eps):
    x, r, rscale, w, dy, dr = _f64(x, r, rscale, w, dy, dr)
    dres = norm_vjp(r, dy * (1.0 if w is None else w), kind, eps) + (0.0 if dr is None else dr)
    out = {"dres": dres, "dx": alpha * dres * (1.0 if rscale is None else rscale),
           "dw": (dy * norm(r, kind, eps)).sum(0)}
    if rscale is not None:
        out["drscale"] = (alpha * x * dres).sum(0)
    return out


def act(z, kind):
    """(act(z), its derivative)."""
    (z,) = _f64(z)
    p = 0.5 * (1.0 + np.tanh(0.5 * z))
    dp = 0.25 / np.cosh(0.5 * np.clip(z, -600, 600)) ** 2
    return (p, dp) if kind == "sigmoid" else (z * p, p + z * dp)


def headnorm_fwd(o, z, w, act_kind, kind, eps):
    o, z, w = _f64(o, z, w)
    y = norm(o, kind, eps).transpose(0, 2, 1, 3) * (1.0 if w is None else w)
    return y if z is None else y * act(z, act_kind)[0]


def headnorm_bwd(o, z, w, dy, act_kind, kind, eps):
    o, z, w, dy = _f64(o, z, w, dy)
    n = norm(o, kind, eps).transpose(0, 2, 1, 3)
    f, df = (1.0, 0.0) if z is None else act(z, act_kind)
    wv = 1.0 if w is None else w
    out = {"do": norm_vjp(o, (dy * f * wv).transpose(0, 2, 1, 3), kind, eps),
           "dz": None if z is None else dy * n * wv * df}
    out["dw"] = None if w is None else (dy * f * n).sum((0, 1) if w.ndim == 2 else (0, 1, 2))
    return out
