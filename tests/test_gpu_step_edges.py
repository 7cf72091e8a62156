"""The ends of a training step on the GPU where they can go wrong.

Tolerances are those of test_gpu_step.py unless a test derives its own."""
import numpy as np
import pytest
import torch

import deterministic_attention_gb300 as da
from oracle import step as os_
from test_gpu_step import BF, F32, _ce_check, _ce_inputs, _done, _f, _gen, _muon_grad

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ cross entropy: loss
def _exact_logits(z):
    """Inputs whose logits are the columns' bf16 numbers exactly: every row of x has a
    single 1.  z [V, N] -> (x, w, z as they are)."""
    w = torch.tensor(z).to(BF)
    return torch.eye(z.shape[1]).to(BF), w, w.double().numpy().T


def _loss_of(z, t):
    """ln(1 + sum over the other words of exp(z - z_target)), which does not cancel."""
    d = z - z[np.arange(len(t)), t][:, None]
    d[np.arange(len(t)), t] = -np.inf
    return np.logaddexp(0.0, np.logaddexp.reduce(d, axis=1))


def _loss_check(z, t, tol):
    x, w, z = _exact_logits(z)
    loss, lse = da.linear_ce_fwd(x.cuda(), w.cuda(), torch.tensor(t, dtype=torch.int32).cuda())
    _done()
    want = _loss_of(z, t)
    assert (_f(loss) >= 0).all(), _f(loss).min()
    assert np.abs(_f(loss) - want).max() <= tol
    at = z[np.arange(len(t)), t]
    assert (np.abs(_f(lse) - (at + want)) <= tol + 2.0 ** -23 * np.abs(at + want)).all()


@pytest.mark.parametrize("lo,hi", [(1.0, 20.0), (40.0, 60.0), (100.0, 400.0), (-300.0, -50.0)])
def test_loss_of_sure_rows(lo, hi):
    """One logit far above the rest, in every group of 32 words of a part of 128.  The
    sum is its own exponential, 1 (2^-22 off), and a correction of the exponents' base
    (an exponential 2^-22 off, two products): 2^-22 + 2^-22 + 2^-23, and ln of a number
    next to 1 adds nothing: 6e-7."""
    rng = np.random.default_rng(0)
    N, V = 512, 700
    z = rng.uniform(-1.0, 1.0, size=(V, N))
    top = rng.uniform(lo, hi, size=N)
    t = np.array([0, 31, 32, 63, 64, 96, 127, 128, 300, 640, 699])[np.arange(N) % 11]
    z += (top - 41.0)[None]
    z[t, np.arange(N)] = top
    _loss_check(z, t, 1e-6)


def test_loss_of_rows_with_several_large_logits():
    """Equal largest logits in several groups, and largest logits that grow from group to
    group: each group scales the sum once more (2^-22 each, and as much for the
    correction, the exponentials and the logarithm's unit of a loss below 2)."""
    rng = np.random.default_rng(1)
    N, V = 512, 384
    top = rng.uniform(16.0, 31.0, size=N)
    z = np.broadcast_to(top - 40.0, (V, N)).copy()
    for i in range(N):
        k = i % 4
        if i < 256:
            z[[5 + 32 * j for j in range(k + 1)], i] = top[i]
        else:
            z[[5, 40, 70, 100], i] = top[i] + np.array([[0, .25, .5, 1], [1, 0, 1, 0], [0, 0, 0, 1], [0, 1, 1, 1]][k])
    _loss_check(z, np.full(N, 5), 8 * 2.0 ** -22)


# ------------------------------------------------------------ cross entropy: gradients
@pytest.mark.parametrize("dloss,dlse", [(1e-38, 10.0), (1e-42, 1e-2), (1e-30, 1e15), (0.0, 1e3), (1e30, 1e-20)])
def test_linear_ce_gradients_of_very_different_size(dloss, dlse):
    """dlse / dloss past fp32's range, or next to it."""
    x, w, t = _ce_inputs(200, 64, 300, seed=3)
    g = _gen(4)
    _ce_check(x, w, t, dloss * torch.rand((200,), generator=g), dlse=dlse * (0.1 + torch.rand((200,), generator=g)),
              dw_fp32=True)


@pytest.mark.parametrize("N,d,V", [(4096, 16, 400001), (1400100, 8, 1000)])
def test_linear_ce_over_more_than_two_pieces(N, d, V):
    """A middle piece's share of dx is added to the sum and kept: four pieces whose tiles of
    dx are all cut along the words, and four of 256 words whose tiles are whole."""
    x, w, t, g = (a.cuda() for a in (*_ce_inputs(N, d, V, seed=6, std=0.2), torch.full((N,), 1.0 / N)))
    _, lse = da.linear_ce_fwd(x, w, t)
    dx, dw = da.linear_ce_bwd(x, w, t, lse, g, dw_fp32=True)
    _done()
    X, W, rows = x.double(), w.double(), max(1, (1 << 28) // V)
    ew = torch.zeros_like(W)
    num = den = worst = worst_lse = 0.0
    for r in range(0, N, rows):
        z = X[r:r + rows] @ W.t()
        top = torch.logsumexp(z, dim=1)
        worst_lse = max(worst_lse, float((lse[r:r + rows] - top).abs().max()))
        p = z.sub_(top[:, None]).exp_().div_(N)
        tr = t[r:r + rows].long()
        p[tr < 0] = 0
        has = (tr >= 0).nonzero()[:, 0]
        p[has, tr[has]] -= 1.0 / N
        ex = p @ W
        ew += p.t() @ X[r:r + rows]
        num += float((dx[r:r + rows] - ex).square().sum())
        den += float(ex.square().sum())
        rms = float(ex.square().mean().sqrt())
        worst = max(worst, float(((dx[r:r + rows] - ex).abs() / ex.abs().clamp(min=rms)).max()))
    assert worst_lse <= 1e-5
    assert (num / den) ** 0.5 <= 2.0 ** -8 and worst <= 2.0 ** -5
    assert float((dw - ew).norm() / ew.norm()) <= 2.0 ** -8


# ------------------------------------------------------------ orthogonalised update
@pytest.mark.parametrize("shape", [(64, 72), (72, 64), (300, 280)])
@pytest.mark.parametrize("s", [3.9, 4.1, 9.0, 15.9])
def test_muon_update_of_large_singular_values(s, shape):
    """One entry, carried to s and back: X, P and X again are each off by 2^-11 at
    most, the result by 2^-8."""
    g = torch.zeros(shape)
    g[5, 7] = -2.0
    o = da.muon_update(g.cuda(), steps=2, coeffs=[(s, 0.0, 0.0), (1.0 / s, 0.0, 0.0)])
    _done()
    want = torch.zeros(shape)
    want[5, 7] = -1.0
    assert np.abs(_f(o) - want.numpy()).max() <= 2.0 ** -8 + 4.1 * 2.0 ** -11


@pytest.mark.parametrize("shape", [(64, 72), (72, 64)])
def test_muon_update_of_large_singular_values_and_their_products(shape):
    """All singular values 5, then through a quintic.  A's rounding (2^-11 of 25) goes into
    P = 0.5 - 0.3125 + 0.0625 as 0.44 2^-11, 1.8 2^-11 of it; P's own and X's three are 2^-11
    each, the result's 2^-8: below 2^-7 in all."""
    q, _ = np.linalg.qr(np.random.default_rng(2).normal(size=(72, 64)))
    g = torch.tensor(q if shape[0] > shape[1] else q.T, dtype=F32).contiguous()
    c = [(40.0, 0.0, 0.0), (0.5, -0.0125, 0.0001)]
    o = da.muon_update(g.cuda(), steps=2, coeffs=c)
    _done()
    want, _ = os_.muon(_f(g), steps=2, coeffs=c)
    assert np.linalg.norm(_f(o) - want) <= 2.0 ** -7 * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(96, 160), (1024, 520)])
def test_muon_update_of_gradients_below_eps(shape, dtype):
    """|u| down to eps / 1024 keeps the accuracy: entries of X are held to 2^-37 at worst,
    2^-37 sqrt(m n) in all against |X| = 2^-10 (7e-6 of 1024 x 520).  Below, that is
    the error of X, times 3.4445 a step."""
    eps = 1e-7
    n = shape[0] * shape[1]
    g = _muon_grad(shape, 50, dtype, eps / 1000 / n ** 0.5)
    o = da.muon_update(g.cuda(), eps=eps)
    tiny = _muon_grad(shape, 51, dtype, 1e-20)
    o2 = da.muon_update(tiny.cuda(), eps=eps)
    _done()
    want, _ = os_.muon(_f(g), eps=eps)
    assert np.linalg.norm(_f(o) - want) <= 2.0 ** -8 * np.linalg.norm(want)
    want, _ = os_.muon(_f(tiny), eps=eps)
    assert np.linalg.norm(_f(o2) - want) <= 3.4445 ** 5 * 2.0 ** -37 * n ** 0.5 * 1.01


# ------------------------------------------------------------ waits
def test_every_wait_of_the_step_operators_runs_out():
    """The self-test's ten waits, one after another, the update's waits for other blocks'
    tiles and for its producer among them: each lasts its limit."""
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    da.selftest_wait_timeout(1_000_000)
    torch.cuda.synchronize()
    with pytest.raises(da.DetAttnError):
        da.check_status()
    a.record()
    da.selftest_wait_timeout(20_000_000)
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) >= 10 * 20.0
    with pytest.raises(da.DetAttnError, match="linear_ce 1, muon_update 1"):
        da.check_status()
    da.check_status()
