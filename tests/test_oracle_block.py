"""Self-tests of oracle/block.py: gradients against central differences, and
the 8-bit format against its definition, spelled out value by value."""
import numpy as np
import pytest

from oracle import block as ob


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("post,pre,gate,as_sigmoid", [
    (True, True, "channel", False), (True, True, "row", True), (False, True, "seq", False),
    (True, False, None, False), (False, True, "seq", True), (True, True, None, False)])
def test_norm_gradients_match_differences(post, pre, gate, as_sigmoid):
    g = _rng(3)
    rows, d, r, s, eps = 6, 8, 0.9, 0.7, 1e-5
    x, y = g.normal(size=(rows, d)), g.normal(size=(rows, d))
    w_post = g.normal(size=d) + 1 if post else None
    w_pre = g.normal(size=d) + 1 if pre else None
    G = {"channel": 1, "seq": 2, "row": rows}.get(gate)
    gt = g.normal(size=(G, d)) if gate else None
    cx, ch = g.normal(size=(rows, d)), g.normal(size=(rows, d))

    def loss(x, y, gt, w_post, w_pre):
        o = ob.norm_fwd(x, y, gt, w_post, w_pre, r, s, eps, as_sigmoid)
        return (o["x"] * cx).sum() + ((o["h"] * ch).sum() if pre else 0.0)

    o = ob.norm_fwd(x, y, gt, w_post, w_pre, r, s, eps, as_sigmoid)
    got = ob.norm_bwd(cx, ch if pre else None, o.get("xhat"), o["yhat"], o.get("rstd_pre"),
                      o.get("rstd_post"), gt, w_post, w_pre, r, s, as_sigmoid)
    args = [x, y, gt, w_post, w_pre]
    for i, name in enumerate(("dx", "dy", "dgate", "dw_post", "dw_pre")):
        if args[i] is None:
            assert name not in got
            continue
        num = np.zeros_like(args[i])
        for at in np.ndindex(*args[i].shape):
            hi, lo = [a if a is None else a.copy() for a in args], [a if a is None else a.copy() for a in args]
            hi[i][at] += 1e-5
            lo[i][at] -= 1e-5
            num[at] = (loss(*hi) - loss(*lo)) / 2e-5
        # Central differences: error h^2 f''' / 6 ~ 1e-10 and rounding 1e-16 / 1e-5 of the loss.
        np.testing.assert_allclose(got[name], num, rtol=1e-6, atol=1e-7)
        assert np.all(got["|%s|" % name] >= np.abs(got[name]) * (1 - 1e-12))


def test_norm_without_block_is_the_plain_norm():
    g = _rng(4)
    x, w, ch = g.normal(size=(3, 8)), g.normal(size=8), g.normal(size=(3, 8))
    o = ob.norm_fwd(x, w_pre=w)
    np.testing.assert_allclose((o["xhat"] ** 2).mean(-1), 1.0, rtol=1e-5)
    got = ob.norm_bwd(np.zeros((3, 8)), ch, o["xhat"], None, o["rstd_pre"], None, w_pre=w, block=False)
    # The norm does not change with the row's scale (but for eps): dx . x = 0.
    np.testing.assert_allclose((got["dx"] * x).sum(-1), 0.0, atol=1e-5)
    assert "dy" not in got


def test_swiglu_gradient_matches_differences():
    g = _rng(5)
    u, dh = g.normal(size=(4, 10)), g.normal(size=(4, 5))
    num = np.zeros_like(u)
    for at in np.ndindex(*u.shape):
        hi, lo = u.copy(), u.copy()
        hi[at] += 1e-5
        lo[at] -= 1e-5
        num[at] = ((ob.swiglu(hi) - ob.swiglu(lo)) * dh).sum() / 2e-5
    np.testing.assert_allclose(ob.swiglu_grad(dh, u), num, rtol=1e-6, atol=1e-8)


def test_act8_follows_its_definition():
    g = _rng(6)
    x = g.normal(size=(40, 64)) * 2.0 ** g.integers(-140, 100, size=(40, 1))
    x[0] = 0.0
    x[1, :32] = 127.0          # exactly representable: k = 0
    x[1, 32:] = 127.0 + 2.0 ** -7  # just past: k = 1
    x[2, 5] = np.inf
    x[3, 40] = np.nan
    q, e = q0, e0 = ob.act8(x)
    for r in range(x.shape[0]):
        for c in range(2):
            v = x[r, 32 * c:32 * c + 32]
            if not np.all(np.isfinite(v)):
                assert e[r, c] == 255 and not q[r, 32 * c:32 * c + 32].any()
                continue
            k = -126
            while np.abs(v).max() > 127.0 * 2.0 ** k:
                k += 1
            assert e[r, c] == k + 127
            want = [int(np.rint(t / 2.0 ** k)) for t in v]
            assert q[r, 32 * c:32 * c + 32].tolist() == want
            assert max(abs(t) for t in want) <= 127
            vals = ob.act8_values(q[r:r + 1], e[r:r + 1])[0, 32 * c:32 * c + 32]
            assert np.all(np.abs(vals - v) <= 2.0 ** (k - 1))
    q, e = ob.act8(np.full((1, 32), 255.0 * 2.0 ** 120))  # the largest bf16 number
    assert (q == 63).all() and (e == 249).all()
    assert e0[1, 0] == 127 and e0[1, 1] == 128 and e0[0, 0] == 1
    assert np.isnan(ob.act8_values(q0, e0)[2, :32]).all()
