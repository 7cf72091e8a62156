"""fp64 oracle of what surrounds an attention layer: norms before and after a
block with gate and residual scale, 8-bit activation checkpoints, the gated
unit, and their closed-form gradients.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``: plain numpy, written
from the formulas, shares no code with the kernels.

RustingBrain vs PyTorch/TensorFlow page, "The setup": a decoder-only model
with RMSNorm and SwiGLU (the page gives neither formula; these are the usual
ones).  Norms divide by the root of the mean square plus eps:

    yhat = y rstd_y,  z = yhat w_post,  x' = r x + s g z
    xhat = x' rstd_x,  h = xhat w_pre

A checkpoint stores, for every 32 consecutive columns of a row, the smallest
k >= -126 with |value| <= 127 2^k, and value / 2^k rounded to even (at k = 122
kept within 63: 64 2^122 is past the largest fp32 and bf16 number).
"""
from __future__ import annotations

import numpy as np

GROUP = 32


def f64(a):
    return np.asarray(a, dtype=np.float64)


# ------------------------------------------------------------ checkpoints
def act8_exponents(x):
    """k per group, int [rows, d / 32]; 128 marks a group that is not finite."""
    x = f64(x)
    rows, d = x.shape
    with np.errstate(invalid="ignore"):
        m = np.abs(x).reshape(rows, d // GROUP, GROUP).max(axis=-1)
    bad = ~np.isfinite(m)
    f, p = np.frexp(np.where(bad, 0.0, m))  # m = f 2^p, f in [1/2, 1)
    k = np.maximum(p - 7 + (f > 127.0 / 128.0), -126)
    k = np.where(m == 0.0, -126, k)
    return np.where(bad, 128, k).astype(np.int64)


def act8(x):
    """(q int8 [rows, d], e uint8 [rows, d / 32]) of x."""
    x = f64(x)
    k = act8_exponents(x)
    kk = np.repeat(k, GROUP, axis=1)
    with np.errstate(invalid="ignore"):
        q = np.where(kk == 128, 0.0, np.rint(np.ldexp(np.where(kk == 128, 0.0, x), -kk)))
    q = np.where(kk == 122, np.clip(q, -63, 63), q)
    return q.astype(np.int8), (k + 127).astype(np.uint8)


def act8_values(q, e):
    k = np.repeat(np.asarray(e, dtype=np.int64) - 127, GROUP, axis=-1)
    return np.where(k == 128, np.nan, np.ldexp(f64(q), np.minimum(k, 127)))


# ------------------------------------------------------------ gated unit
def sigmoid(a):
    a = f64(a)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-a))


def swiglu(u):
    a, b = np.split(f64(u), 2, axis=-1)
    return a * sigmoid(a) * b


def swiglu_grad(dh, u):
    a, b = np.split(f64(u), 2, axis=-1)
    s, dh = sigmoid(a), f64(dh)
    return np.concatenate([dh * b * s * (1.0 + a * (1.0 - s)), dh * a * s], axis=-1)


# ------------------------------------------------------------ block norms
def rstd(x, eps):
    x = f64(x)
    return 1.0 / np.sqrt((x * x).mean(axis=-1) + eps)


def gate_rows(gate, rows, as_sigmoid):
    """The gate of every row, [rows, d] (ones without a gate)."""
    if gate is None:
        return 1.0
    g = sigmoid(gate) if as_sigmoid else f64(gate)
    return np.repeat(g, rows // g.shape[0], axis=0)


def norm_fwd(x, y=None, gate=None, w_post=None, w_pre=None, r=1.0, s=1.0, eps=1e-6,
             as_sigmoid=False):
    """Everything a forward gives, as a dict (what it does not give is absent)."""
    x, out = f64(x), {}
    if y is not None:
        yhat = f64(y)
        if w_post is not None:
            out["rstd_post"] = rstd(yhat, eps)
            yhat = yhat * out["rstd_post"][:, None]
        out["yhat"] = yhat
        z = yhat * f64(w_post) if w_post is not None else yhat
        x = r * x + s * gate_rows(gate, x.shape[0], as_sigmoid) * z
    out["x"] = x
    if w_pre is not None:
        out["rstd_pre"] = rstd(x, eps)
        out["xhat"] = x * out["rstd_pre"][:, None]
        out["h"] = out["xhat"] * f64(w_pre)
    return out


def norm_bwd(dx_out, dh, xhat, yhat, rstd_pre, rstd_post, gate=None, w_post=None, w_pre=None,
             r=1.0, s=1.0, as_sigmoid=False, block=True):
    """Gradients as a dict, from the normed values and row statistics; every
    entry "|name|" is the sum of the magnitudes that make up "name"."""
    out = {}
    D, mag = f64(dx_out), np.abs(f64(dx_out))
    rows, d = D.shape
    if w_pre is not None:
        dh, xhat, rp = f64(dh), f64(xhat), f64(rstd_pre)[:, None]
        a = dh * f64(w_pre)
        D = D + rp * (a - xhat * (a * xhat).mean(axis=-1, keepdims=True))
        mag = mag + rp * (np.abs(a) + np.abs(xhat) * np.abs(a * xhat).mean(axis=-1, keepdims=True))
        out["dw_pre"] = (dh * xhat).sum(axis=0)
        out["|dw_pre|"] = np.abs(dh * xhat).sum(axis=0)
    if not block:
        out["dx"], out["|dx|"] = D, mag
        return out
    out["dx"], out["|dx|"] = r * D, abs(r) * mag
    g = gate_rows(gate, rows, as_sigmoid)
    dz, mag = s * g * D, np.abs(s * g) * mag
    if gate is not None or w_post is not None:
        yhat = f64(yhat)
    w = f64(w_post) if w_post is not None else 1.0
    if gate is not None:
        # sigma' = sigma(x) sigma(-x): 1 - sigma has no digits left for large x.
        slope = g * gate_rows(-f64(gate), rows, True) if as_sigmoid else np.ones_like(g)
        G = np.asarray(gate).shape[0]
        t = s * D * yhat * w * slope
        tm = np.abs(out["|dx|"] / max(abs(r), 1e-300) * s * yhat * w * slope) if r else np.abs(t)
        out["dgate"] = t.reshape(G, rows // G, d).sum(axis=1)
        out["|dgate|"] = tm.reshape(G, rows // G, d).sum(axis=1)
    if w_post is not None:
        ro = f64(rstd_post)[:, None]
        out["dw_post"], out["|dw_post|"] = (dz * yhat).sum(axis=0), (mag * np.abs(yhat)).sum(axis=0)
        a, am = dz * w, mag * np.abs(w)
        dz = ro * (a - yhat * (a * yhat).mean(axis=-1, keepdims=True))
        mag = ro * (am + np.abs(yhat) * (am * np.abs(yhat)).mean(axis=-1, keepdims=True))
    out["dy"], out["|dy|"] = dz, mag
    return out
