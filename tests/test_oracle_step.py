"""Pins of the oracle of the ends of a training step, and of rope_freqs (host
only).  No GPU needed."""
import math

import numpy as np
import pytest

import deterministic_attention_gb300 as da
from oracle import step as os_


def test_rope_turns_a_pair_by_its_angle():
    f = np.array([0.5, 0.25])
    x = np.zeros((3, 1, 6))
    x[:, 0, 0] = 1.0            # pair 0 in both layouts, first component
    x[:, 0, 4:] = 7.0           # behind the turned part
    for inter, second in ((False, 2), (True, 1)):
        y = os_.rope(x, np.arange(3), f, inter, mscale=2.0)
        np.testing.assert_allclose(y[:, 0, 0], 2 * np.cos(0.5 * np.arange(3)))
        np.testing.assert_allclose(y[:, 0, second], 2 * np.sin(0.5 * np.arange(3)))
        np.testing.assert_array_equal(y[:, 0, 4:], 7.0)
        np.testing.assert_allclose(os_.rope(y, np.arange(3), f, inter, 0.5, back=True), np.where(
            np.arange(6) < 4, x, x), atol=1e-15)


def test_rope_scores_depend_on_distance_alone():
    rng = np.random.default_rng(0)
    q, k, f = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8)), 10.0 ** -np.arange(4)
    dot = [float((os_.rope(q, [t], f) * os_.rope(k, [t - 5], f)).sum()) for t in (5, 17, 4096)]
    np.testing.assert_allclose(dot, dot[0], rtol=1e-12)


def test_cross_entropy_of_known_logits():
    w = np.eye(4)
    x = np.log(np.array([[1.0, 2.0, 3.0, 4.0], [1.0, 1.0, 1.0, 1.0]]))
    loss, lse, p = os_.linear_ce(x, w, [3, -1])
    np.testing.assert_allclose(loss, [math.log(10 / 4), 0.0], atol=1e-15)
    np.testing.assert_allclose(lse, [math.log(10), math.log(4)])
    np.testing.assert_allclose(p[0], [0.1, 0.2, 0.3, 0.4])


@pytest.mark.parametrize("planted", [False, True])
def test_cross_entropy_gradient_against_differences(planted):
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(5, 3)), rng.normal(size=(7, 3))
    t, g, e = np.array([0, 6, -1, 3, 3]), rng.normal(size=5), rng.normal(size=5)
    f = lambda x, w: float((g * os_.linear_ce(x, w, t)[0]).sum() + (e * os_.linear_ce(x, w, t)[1]).sum())
    dx, dw, _, _ = os_.linear_ce_grad(x, w, t, g if not planted else 1.01 * g, e)
    worst = 0.0
    for a, da_, which in ((x, dx, 0), (w, dw, 1)):
        for i in np.ndindex(a.shape):
            h = np.zeros_like(a)
            h[i] = 1e-5
            args = ((x + h, w), (x - h, w)) if which == 0 else ((x, w + h), (x, w - h))
            worst = max(worst, abs((f(*args[0]) - f(*args[1])) / 2e-5 - da_[i]))
    assert (worst > 1e-4) if planted else (worst < 1e-8)


@pytest.mark.parametrize("m,n", [(4, 9), (9, 4), (6, 6)])
def test_muon_is_the_polynomial_of_the_singular_values(m, n):
    g = np.random.default_rng(2).normal(size=(m, n))
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / np.sqrt((s * s).sum())
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    o, mom = os_.muon(g, eps=0.0)
    assert mom is None
    np.testing.assert_allclose(o, (u * s) @ vt, atol=1e-12)


def test_muon_momentum():
    g, m = np.ones((2, 8)), np.full((2, 8), 2.0)
    o, m1 = os_.muon(g, m, beta=0.5, steps=1)
    np.testing.assert_array_equal(m1, 2.0)
    np.testing.assert_allclose(o, os_.muon(g + 0.5 * m1, steps=1)[0])
    np.testing.assert_allclose(os_.muon(g, m, beta=0.5, nesterov=False)[0], os_.muon(m1)[0])


# ------------------------------------------------------------ rope_freqs
def _freqs(*a, **k):
    f, m = da.rope_freqs(*a, device="cpu", **k)
    return f.numpy(), m


def test_rope_freqs_plain_linear_and_base():
    da.build()
    i = np.arange(32)
    f, m = _freqs(64)
    assert m == 1.0
    np.testing.assert_allclose(f, 10000.0 ** (-i / 32.0), rtol=1e-14)
    np.testing.assert_allclose(_freqs(64, scaling="linear", factor=8.0)[0], f / 8.0, rtol=1e-14)
    s, _ = _freqs(64, scaling="base", factor=8.0)
    assert s[0] == 1.0
    np.testing.assert_allclose(s[-1], f[-1] / 8.0, rtol=1e-12)  # the slowest pair is interpolated
    np.testing.assert_allclose(s, (10000.0 * 8.0 ** (64 / 62)) ** (-i / 32.0), rtol=1e-13)


def test_rope_freqs_bands():
    f, _ = _freqs(128, base=500000.0)
    s, m = _freqs(128, base=500000.0, scaling="bands", factor=8.0, context=8192)
    turns = 8192 * f / (2 * np.pi)
    assert m == 1.0
    np.testing.assert_array_equal(s[turns > 4], f[turns > 4])
    np.testing.assert_allclose(s[turns < 1], f[turns < 1] / 8, rtol=1e-14)
    mid = (turns >= 1) & (turns <= 4)
    k = (turns[mid] - 1) / 3
    assert mid.any()
    np.testing.assert_allclose(s[mid], f[mid] * (k + (1 - k) / 8), rtol=1e-13)


def test_rope_freqs_ramp():
    f, _ = _freqs(128)
    s, m = _freqs(128, scaling="ramp", factor=16.0, context=4096)
    assert abs(m - (0.1 * math.log(16.0) + 1.0)) < 1e-6
    at = lambda turns: 128 * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
    lo, hi = math.floor(at(32.0)), math.ceil(at(1.0))
    k = 1 - np.clip((np.arange(64) - lo) / (hi - lo), 0, 1)
    np.testing.assert_allclose(s, f * (k + (1 - k) / 16), rtol=1e-13)
    assert s[0] == f[0] and abs(s[-1] / f[-1] - 1 / 16) < 1e-12


def test_rope_freqs_ramp_of_a_context_shorter_than_a_turn():
    f, _ = _freqs(64)
    s, _ = _freqs(64, scaling="ramp", factor=4.0, context=4)
    assert s[0] == f[0]
    np.testing.assert_allclose(s[1:], f[1:] / 4, rtol=1e-14)
