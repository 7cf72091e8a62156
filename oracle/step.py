"""fp64 oracle of the ends of a training step: rotary positions, the output
projection's softmax cross entropy, the orthogonalised update.  Plain numpy,
written from the definitions in include/detattn.h."""
from __future__ import annotations

import numpy as np

NS = (3.4445, -4.7750, 2.0315)


def rope(x, positions, freqs, interleaved=False, mscale=1.0, back=False):
    """x [..., T, H, D], positions [..., T]: the first 2 len(freqs) components turned."""
    x = np.array(x, np.float64)
    n = len(freqs)
    angle = np.multiply.outer(np.asarray(positions, np.float64), np.asarray(freqs, np.float64))
    turn = mscale * np.exp((-1j if back else 1j) * angle)[..., None, :]
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = (x[..., a] + 1j * x[..., b]) * turn
    x[..., a], x[..., b] = z.real, z.imag
    return x


def linear_ce(x, w, targets):
    """(loss [N], lse [N], p [N, V])."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(axis=1, keepdims=True)
    t = np.asarray(targets)
    zt = z[np.arange(len(t)), np.maximum(t, 0)]
    loss = np.where(t >= 0, (top[:, 0] - zt) + np.log(s[:, 0]), 0.0)
    return loss, (top + np.log(s))[:, 0], e / s


def linear_ce_grad(x, w, targets, dloss, dlse=None):
    """(dx, dw, dz, p)."""
    _, _, p = linear_ce(x, w, targets)
    t = np.asarray(targets)
    g = np.where(t >= 0, np.asarray(dloss, np.float64), 0.0)
    dz = p * (g + (0.0 if dlse is None else np.asarray(dlse, np.float64)))[:, None]
    rows = np.arange(len(t))[t >= 0]
    dz[rows, t[rows]] -= g[rows]
    return dz @ np.asarray(w, np.float64), dz.T @ np.asarray(x, np.float64), dz, p


def _keep(v, _):
    return v


def to_fp16(v, scale):
    """v rounded as fp16 holds it after multiplication by a power of two."""
    return (v * scale).astype(np.float16).astype(np.float64) / scale


def muon(g, momentum=None, beta=0.95, nesterov=True, steps=5, coeffs=None, eps=1e-7, rounding=_keep):
    """(update, momentum) of one matrix.  rounding(values, scale) is applied to
    what the products pass on: with to_fp16, the size of the error that holding
    those in fp16 leaves."""
    u = np.asarray(g, np.float64)
    if momentum is not None:
        momentum = beta * np.asarray(momentum, np.float64) + u
        u = u + beta * momentum if nesterov else momentum
    x = rounding(u / (np.sqrt((u * u).sum()) + eps), 4096.0)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for k in range(steps):
        a, b, c = NS if coeffs is None else coeffs[k]
        gram = rounding(x @ x.T, 128.0)
        p = rounding(a * np.eye(len(x)) + b * gram + c * (gram @ gram), 1024.0)
        x = p @ x
        if k < steps - 1:
            x = rounding(x, 4096.0)
    return (x.T if tall else x), momentum
