"""The ends of a training step on the GPU against the fp64 oracle: rotary
positions, the output projection's cross entropy, the orthogonalised update.

Tolerances.  A bf16 result is off by half a step, 2^-8 of the value at most, an
fp16 number by 2^-11, an fp32 one by 2^-24.  A tensor core adds K products of
bf16 numbers (exact in fp32) in K / 16 instructions; each loses at most one
step (2^-23) of what it adds to and, aligning its sixteen products, of the
largest one: (K / 16 + 16) 2^-23 sum |a b| in all."""
import numpy as np
import pytest
import torch

import deterministic_attention_gb300 as da
from oracle import step as os_

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    da.build()
    da.lib()


def _f(t):
    return t.detach().cpu().double().numpy()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _sums(K):
    return (K / 16 + 16) * 2.0 ** -23


def _done():
    torch.cuda.synchronize()
    da.check_status()


# ------------------------------------------------------------ rotary positions
def _rope_tol(x, want, m, dtype):
    """cos and sin: the phase's rounding to 24 bits (2^-25 of half a turn, 1e-7)
    and sincospi's two units, 2^-22 in all; three fp32 operations; the result's rounding."""
    pairs = np.abs(x).max(axis=-1, keepdims=True)  # |a| + |b| <= 2 max
    return 2 * m * pairs * 2.0 ** -21 + np.abs(want) * (2.0 ** -8 if dtype is BF else 2.0 ** -24)


def _rope_case(B, T, Hq, Hkv, D, rot, inter, dtype, positions=None, joined=False, scaling=None, seed=0, back=False):
    g = _gen(seed)
    qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=g).to(dtype).cuda()
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    if not joined:
        q, k = q.contiguous(), k.contiguous()
    f, m = da.rope_freqs(rot, scaling=scaling, factor=8.0, context=4096)
    call = da.rope_bwd if back else da.rope_fwd
    qo, ko = call(q, k, f, positions=None if positions is None else positions.cuda(), interleaved=inter, mscale=m)
    _done()
    t = np.broadcast_to(np.arange(T) if positions is None else positions.numpy(), (B, T))
    for x, y in ((q, qo), (k, ko)):
        assert y.is_contiguous() and y.dtype is dtype and y.shape == x.shape
        want = os_.rope(_f(x), t, _f(f), inter, m, back)
        assert (np.abs(_f(y) - want) <= _rope_tol(_f(x), want, m, dtype)).all()
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot", [
    (1, 1, 1, 1, 64, 64), (2, 33, 3, 1, 64, 64), (2, 40, 4, 2, 128, 64), (1, 129, 5, 5, 128, 32),
    (3, 7, 2, 1, 80, 40), (2, 9, 1, 1, 66, 6), (1, 5, 2, 1, 128, 2), (1, 3, 1, 1, 2, 2), (1, 2, 1, 1, 1024, 1024),
    (1, 1500, 12, 4, 64, 64), (1, 17, 40, 8, 96, 48)])
def test_rope(B, T, Hq, Hkv, D, rot, dtype, inter):
    _rope_case(B, T, Hq, Hkv, D, rot, inter, dtype)
    _rope_case(B, T, Hq, Hkv, D, rot, inter, dtype, joined=True, back=True, seed=1)


@pytest.mark.parametrize("scaling", [None, "linear", "base", "ramp", "bands"])
def test_rope_far_positions(scaling):
    p = torch.tensor([[0, 1, 131071, 1 << 24, (1 << 31) - 1], [-1, -(1 << 31), 1048575, 7, 99999]], dtype=torch.int32)
    # (the oracle's angle in doubles: 2^31 steps of 2^-53 of it are 2^-21 radians)
    _rope_case(2, 5, 2, 1, 128, 128, False, F32, positions=p, scaling=scaling)
    _rope_case(2, 5, 2, 1, 128, 64, True, BF, positions=p, scaling=scaling, joined=True)


def test_rope_positions_of_one_sequence_serve_all():
    _rope_case(3, 4, 2, 1, 64, 64, False, BF, positions=torch.tensor([5, 0, 9, 2], dtype=torch.int32))


def test_rope_one_pair_over_several_blocks_and_turns():
    f = torch.tensor([1e9, 6.283185307179586, 100.0, -0.3], dtype=torch.float64, device="cuda")
    x = torch.randn((1, 700, 1, 8), generator=_gen(3)).cuda()
    y, none = da.rope_fwd(x, None, f)
    _done()
    assert none is None
    # Angles of up to 7e11 radians: the oracle's double is off by 2^-53 of them.
    want = os_.rope(_f(x), np.arange(700)[None], _f(f))
    assert np.abs(_f(y) - want)[..., [1, 2, 3, 5, 6, 7]].max() <= 2e-6 * np.abs(_f(x)).max() * 2
    assert np.abs(_f(y) - want).max() <= 700 * 1e9 * 2.0 ** -53 * 2 * np.abs(_f(x)).max() + 1e-5


@pytest.mark.parametrize("dtype,D,rot", [(BF, 64, 64), (BF, 64, 20), (F32, 66, 6)])
def test_rope_in_place_and_parts(dtype, D, rot):
    """In place in the joined projection: V and what lies around it stay; the same as out of place."""
    f, _ = da.rope_freqs(rot)
    buf = torch.randn((2, 50, 7, D), generator=_gen(4)).to(dtype).cuda()
    q, k = buf[:, :, 1:4], buf[:, :, 4:6]
    before = buf.clone()
    want = da.rope_fwd(q, k, f)
    got = da.rope_fwd(q, k, f, q_out=q, k_out=k)
    _done()
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, :, 0], before[:, :, 0]) and torch.equal(buf[:, :, 6], before[:, :, 6])
    out = torch.full((2, 50, 9, D), 3.0, dtype=dtype, device="cuda")
    da.rope_bwd(q, k, f, dq_out=out[:, :, 5:8], dk_out=out[:, :, 2:4])
    _done()
    for h in (0, 1, 4, 8):
        assert (out[:, :, h] == 3.0).all()
    assert (out[:, :, 5:8] - before[:, :, 1:4]).abs().max() <= (0.05 if dtype is BF else 1e-5)


@pytest.mark.parametrize("dtype,offset", [(BF, 1), (BF, 2), (BF, 4), (F32, 1), (F32, 2)])
def test_rope_from_any_element(dtype, offset):
    """Tensors that begin on any element: narrower vectors, the same numbers, nothing around them."""
    f, _ = da.rope_freqs(32)
    n = 2 * 30 * 3 * 64
    q = torch.randn((2, 30, 3, 64), generator=_gen(50)).to(dtype).cuda()
    src, dst = (torch.full((n + 16,), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    src[offset:offset + n] = q.view(-1)
    for inter in (False, True):
        want, _ = da.rope_fwd(q, None, f, interleaved=inter)
        got, _ = da.rope_fwd(src[offset:offset + n].view(q.shape), None, f, interleaved=inter,
                             q_out=dst[offset:offset + n].view(q.shape))
        _done()
        assert torch.equal(got, want)
        assert (dst[:offset] == 7).all() and (dst[offset + n:] == 7).all()


def test_rope_bwd_is_the_gradient():
    f, m = da.rope_freqs(64, scaling="ramp", factor=4.0, context=64)
    q, dq = (torch.randn((1, 20, 2, 64), generator=_gen(s)).cuda() for s in (5, 6))
    y, _ = da.rope_fwd(q, None, f, mscale=m)
    dx, _ = da.rope_bwd(dq, None, f, mscale=m)
    _done()
    # <dq, rope q> = <rope^T dq, q>, and differences of the (linear) map itself.
    a, b = (_f(dq) * _f(y)).sum(), (_f(dx) * _f(q)).sum()
    assert abs(a - b) <= 1e-5 * (np.abs(_f(dq)) * np.abs(_f(y))).sum()
    for i in (0, 31, 32, 63):
        e = torch.zeros_like(q)
        e[0, 7, 1, i] = 0.5
        up, down = da.rope_fwd(q + e, None, f, mscale=m)[0], da.rope_fwd(q - e, None, f, mscale=m)[0]
        assert abs((_f(dq) * (_f(up) - _f(down))).sum() - _f(dx)[0, 7, 1, i]) <= 1e-4


def test_rope_refuses_views_it_cannot_walk():
    f, _ = da.rope_freqs(64)
    x = torch.zeros((4, 6, 2, 64), dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="one stride"):
        da.rope_fwd(x[:, :3], None, f)
    with pytest.raises(ValueError, match="contiguous"):
        da.rope_fwd(x.transpose(2, 3), None, f)
    with pytest.raises(ValueError, match="positions"):
        da.rope_fwd(x, None, f, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        da.rope_fwd(x, None, f.float())
    with pytest.raises(TypeError):
        da.rope_fwd(x.half(), None, f)
    with pytest.raises(TypeError):
        da.rope_fwd(x, x[:, :, :1].float(), f)
    with pytest.raises(da.DetAttnError):
        da.rope_fwd(x[..., :32].contiguous(), None, f)      # more components than a head has
    q, k = da.rope_fwd(x[:0], x[:0], f)
    assert q.shape == (0, 6, 2, 64) and k.shape == q.shape


# ------------------------------------------------------------ cross entropy
def _ce_inputs(N, d, V, seed=0, no_target=0.2, std=0.05):
    g = _gen(seed)
    x = torch.randn((N, d), generator=g).to(BF)
    w = (std * torch.randn((V, d), generator=g)).to(BF)
    t = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    t[torch.rand((N,), generator=g) < no_target] = -100
    return x, w, t


def _ce_check(x, w, t, dloss=None, dlse=None, dw_fp32=False, lse=None):
    N, d = x.shape
    V = w.shape[0]
    c = lambda a: None if a is None else a.cuda()
    loss, got_lse = da.linear_ce_fwd(c(x), c(w), c(t))
    _done()
    X, W = _f(x), _f(w)
    want_loss, want_lse, p = os_.linear_ce(X, W, t.numpy())
    mag = (np.abs(X) @ np.abs(W).T).max(axis=1)            # a row's largest sum |x w|
    dz_ = _sums(d) * mag + 2.0 ** -20                      # a logit; the exponentials' and logarithm's few units
    assert (np.abs(_f(got_lse) - want_lse) <= dz_ + 2.0 ** -22 * np.abs(want_lse)).all()
    assert (np.abs(_f(loss) - want_loss) <= 2 * dz_ + 2.0 ** -22 * np.abs(want_loss)).all()
    assert (_f(loss)[t.numpy() < 0] == 0).all()
    if dloss is None:
        return
    dx, dw = da.linear_ce_bwd(c(x), c(w), c(t), got_lse, c(dloss), dlse=c(dlse), dw_fp32=dw_fp32)
    _done()
    assert dw.dtype is (F32 if dw_fp32 else BF) and dx.dtype is BF
    ex, ew, dz, p = os_.linear_ce_grad(X, W, t.numpy(), _f(dloss), None if dlse is None else _f(dlse))
    coef = np.where(t.numpy() >= 0, _f(dloss), 0.0) + (0.0 if dlse is None else _f(dlse))
    # dz: rounded to bf16 after an exponential whose argument carries the
    # logit's and lse's errors.
    off = 2.0 ** -8 * np.abs(dz) + (2 * dz_ + 2.0 ** -20)[:, None] * np.abs(coef)[:, None] * p * 2 + 1e-38
    tx = off @ np.abs(W) + _sums(V) * (np.abs(dz) @ np.abs(W)) + 2.0 ** -8 * np.abs(ex)
    tw = off.T @ np.abs(X) + _sums(N) * (np.abs(dz).T @ np.abs(X)) + 2.0 ** -8 * np.abs(ew)
    assert (np.abs(_f(dx) - ex) <= tx * 1.001).all()
    assert (np.abs(_f(dw) - ew) <= tw * 1.001).all()
    # As a whole: roundings of both kinds are independent, rms 0.42 of half a step each.
    rel = lambda a, b: np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300)
    if N * d > 2000:
        assert rel(_f(dx), ex) <= 2.0 ** -8 and rel(_f(dw), ew) <= 2.0 ** -8


@pytest.mark.parametrize("N,d,V", [
    (1, 8, 1), (1, 64, 2), (2, 8, 255), (255, 64, 256), (256, 72, 257), (257, 64, 129), (129, 264, 1000),
    (300, 768, 513), (700, 8, 5003), (64, 1536, 300)])
def test_linear_ce(N, d, V):
    x, w, t = _ce_inputs(N, d, V, seed=N)
    g = _gen(N + 1)
    _ce_check(x, w, t, torch.rand((N,), generator=g) / N)
    _ce_check(x, w, t, torch.full((N,), 1.0 / 240), dlse=1e-3 * torch.randn((N,), generator=g), dw_fp32=True)


def test_linear_ce_large_logits_and_sure_rows():
    """Rows whose target has nearly all the weight: the loss keeps its digits."""
    x, w, t = _ce_inputs(200, 64, 900, seed=5, no_target=0.0, std=0.3)
    x = (x.float() + 2.0 * w[t.long()].float()).to(BF)
    _ce_check(x, w, t, torch.full((200,), 0.005))
    x[:100] = (8 * x[:100].float()).to(BF)                 # logits of hundreds: most terms underflow
    _ce_check(x, w, t, torch.full((200,), 0.005))


def test_linear_ce_over_several_pieces():
    """More than 1 GiB of dz: two pieces, the last narrower; and a padded vocabulary."""
    N, d, V = 4200, 40, 132001
    x, w, t = _ce_inputs(N, d, V, seed=6, std=0.2)
    g = torch.full((N,), 1.0 / N)
    dev = [a.cuda() for a in (x, w, t, g)]
    loss, lse = da.linear_ce_fwd(*dev[:3])
    dx, dw = da.linear_ce_bwd(*dev[:3], lse, dev[3])
    dx2, dw2 = da.linear_ce_bwd(*dev[:3], lse, dev[3])
    _done()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    X, W = dev[0].double(), dev[1].double()
    z = X @ W.t()
    want = torch.logsumexp(z, dim=1)
    assert float((lse - want).abs().max()) <= 1e-5
    p = torch.exp(z - want[:, None]) / N
    p[dev[2] < 0] = 0
    rows = (dev[2] >= 0).nonzero()[:, 0]
    p[rows, dev[2][rows].long()] -= 1.0 / N
    for a, b in ((dx, p @ W), (dw, p.t() @ X)):
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -8
        assert float(((a - b).abs() / b.abs().clamp(min=float(b.square().mean().sqrt()))).max()) <= 2.0 ** -5


def test_linear_ce_gradient_against_differences():
    """Differences of the loss itself, along directions in x and in w (bf16 inputs: large steps
    that are bf16 numbers, second order removed by the symmetric difference of a smooth sum)."""
    N, d, V = 64, 64, 300
    x, w, t = (a.cuda() for a in _ce_inputs(N, d, V, seed=7, std=0.1))
    g = torch.rand((N,), generator=_gen(8)).cuda()
    _, lse = da.linear_ce_fwd(x, w, t)
    dx, dw = da.linear_ce_bwd(x, w, t, lse, g, dw_fp32=True)
    total = lambda x, w: float((g.double() * da.linear_ce_fwd(x, w, t)[0].double()).sum())
    for i in range(4):
        sx = torch.sign(torch.randn((N, d), generator=_gen(10 + i))).cuda()
        xp, xm = (x.float() + 0.01 * sx).to(BF), (x.float() - 0.01 * sx).to(BF)
        want = float((dx.double() * (xp.double() - xm.double())).sum())
        scale = float((dx.double().abs() * (xp.double() - xm.double()).abs()).sum())
        assert abs(total(xp, w) - total(xm, w) - want) <= 2.0 ** -7 * scale
        sw = torch.sign(torch.randn((V, d), generator=_gen(20 + i))).cuda()
        wp, wm = (w.float() + 0.004 * sw).to(BF), (w.float() - 0.004 * sw).to(BF)
        want = float((dw.double() * (wp.double() - wm.double())).sum())
        scale = float((dw.double().abs() * (wp.double() - wm.double()).abs()).sum())
        assert abs(total(x, wp) - total(x, wm) - want) <= 2.0 ** -7 * scale
    _done()


def test_linear_ce_rows_without_targets():
    x, w, t = _ce_inputs(300, 64, 500, seed=9)
    t[:] = -1
    t[17] = -(1 << 31)
    dev = [a.cuda() for a in (x, w, t)]
    loss, lse = da.linear_ce_fwd(*dev)
    g = torch.full((300,), NAN, device="cuda")             # not read where there is no target
    dx, dw = da.linear_ce_bwd(*dev, lse, g)
    _done()
    assert (loss == 0).all() and torch.isfinite(lse).all() and (dx == 0).all() and (dw == 0).all()
    # lse has its gradient all the same.
    e = torch.full((300,), 0.25)
    _ce_check(x, w, t, torch.zeros(300), dlse=e)
    # A row without a gradient gives zeros although its lse is no number.
    lse[3] = NAN
    dx, dw = da.linear_ce_bwd(*dev, lse, g)
    _done()
    assert (dx == 0).all() and (dw == 0).all()


def test_linear_ce_bad_rows_stay_by_themselves():
    x, w, t = (a.cuda() for a in _ce_inputs(300, 64, 500, seed=11, no_target=0.0))
    loss, lse = da.linear_ce_fwd(x, w, t)
    y = x.clone()
    y[100, 3], y[200, 5] = NAN, INF
    loss2, lse2 = da.linear_ce_fwd(y, w, t)
    g = torch.full((300,), 1e-3, device="cuda")
    dx, _ = da.linear_ce_bwd(x, w, t, lse, g)
    dx2, dw2 = da.linear_ce_bwd(y, w, t, lse2, g)
    _done()
    ok = torch.ones(300, dtype=torch.bool)
    ok[[100, 200]] = False
    assert torch.equal(loss[ok], loss2[ok]) and torch.equal(lse[ok], lse2[ok])
    assert loss2[~ok].isnan().all() and torch.equal(dx[ok], dx2[ok]) and dx2[~ok].isnan().any(dim=1).all()
    assert dw2[:, 3].isnan().all()


def test_linear_ce_reports_targets_past_the_vocabulary():
    x, w, t = (a.cuda() for a in _ce_inputs(40, 64, 500, seed=12, no_target=0.0))
    t2 = t.clone()
    t[5], t[6] = 500, (1 << 31) - 1
    t2[5] = t2[6] = -1
    loss, lse = da.linear_ce_fwd(x, w, t)
    torch.cuda.synchronize()
    with pytest.raises(da.DetAttnError, match="linear_ce"):
        da.check_status()
    g = torch.full((40,), 0.1, device="cuda")
    dx, dw = da.linear_ce_bwd(x, w, t, lse, g)
    torch.cuda.synchronize()
    with pytest.raises(da.DetAttnError, match="linear_ce"):
        da.check_status()
    assert torch.equal(loss, da.linear_ce_fwd(x, w, t2)[0])
    dx2, dw2 = da.linear_ce_bwd(x, w, t2, lse, g)
    _done()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_linear_ce_outputs_workspaces_and_shapes():
    x, w, t = (a.cuda() for a in _ce_inputs(6 * 50, 64, 777, seed=13))
    loss, lse = da.linear_ce_fwd(x.view(6, 50, 64), w, t.view(6, 50))
    assert loss.shape == lse.shape == (6, 50)
    g = torch.full((6, 50), 0.01, device="cuda")
    dx, dw = da.linear_ce_bwd(x.view(6, 50, 64), w, t.view(6, 50), lse, g)
    # Guard bytes around every output, garbage in the workspaces.
    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[32:32 + n].view(shape)
    bufs, outs = zip(*(guarded(s, dt) for s, dt in (((300,), F32), ((300,), F32), ((300, 64), BF), ((777, 64), BF))))
    ws = torch.full((da.linear_ce_fwd_workspace_bytes(300, 777, 64),), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((da.linear_ce_bwd_workspace_bytes(300, 777, 64),), 255, dtype=torch.uint8, device="cuda")
    da.linear_ce_fwd(x, w, t, loss=outs[0], lse=outs[1], workspace=ws)
    da.linear_ce_bwd(x, w, t, outs[1], g.view(-1), dx=outs[2], dw=outs[3], workspace=wb)
    _done()
    for a, b in zip(outs, (loss.view(-1), lse.view(-1), dx.view(300, 64), dw)):
        assert torch.equal(a, b)
    for b in bufs:
        assert (b[:32] == 7).all() and (b[-32:] == 7).all()
    with pytest.raises(da.DetAttnError, match="workspace"):
        da.linear_ce_fwd(x, w, t, workspace=ws[:-1])
    with pytest.raises(da.DetAttnError, match="workspace"):
        da.linear_ce_bwd(x, w, t, lse.view(-1), g.view(-1), workspace=wb[:-1])
    with pytest.raises(TypeError):
        da.linear_ce_fwd(x, w.float(), t)
    with pytest.raises(TypeError):
        da.linear_ce_fwd(x, w, t.long())
    with pytest.raises(ValueError):
        da.linear_ce_fwd(x, w, t[:-1])
    e = x[:0]
    loss, lse = da.linear_ce_fwd(e, w, t[:0])
    dx, dw = da.linear_ce_bwd(e, w, t[:0], lse, lse, dw_fp32=True)
    _done()
    assert loss.numel() == 0 and dx.shape == (0, 64) and dw.shape == (777, 64) and (dw == 0).all()


# ------------------------------------------------------------ orthogonalised update
def _muon_check(g, momentum=None, **kw):
    gd = g.cuda()
    md = None if momentum is None else momentum.cuda()
    o = da.muon_update(gd, momentum=md, **kw)
    _done()
    assert o.dtype is BF and o.shape == g.shape
    m, n = g.shape[-2:]
    for i in np.ndindex(g.shape[:-2]):
        m0 = None if momentum is None else _f(momentum[i])
        want, wm = os_.muon(_f(g[i]), m0, **kw)
        held, _ = os_.muon(_f(g[i]), m0, rounding=os_.to_fp16, **kw)
        if wm is not None:
            assert (np.abs(_f(md[i]) - wm) <= 2.0 ** -22 * (np.abs(wm) + np.abs(_f(g[i])) + np.abs(m0))).all()
        # Twice what holding X, X X^T and P in fp16 leaves (which the oracle
        # forms with the same roundings elsewhere), and the rounding to bf16.
        norm = np.linalg.norm(want)
        off = np.linalg.norm(_f(o[i]) - want)
        assert off <= 2 * np.linalg.norm(held - want) + 2.0 ** -8 * norm + 1e-30, (i, off / norm)


def _muon_grad(shape, seed, dtype, std=1e-3):
    return (std * torch.randn(shape, generator=_gen(seed))).to(dtype)


@pytest.mark.parametrize("shape", [(8, 8), (1, 8), (1, 64), (64, 8), (128, 128), (129, 136), (256, 256), (257, 264),
                                   (300, 520), (520, 304), (3, 100, 72), (2, 3, 72, 200), (1, 768, 768), (5, 8)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_muon_update(shape, dtype):
    g = _muon_grad(shape, 1, dtype)
    _muon_check(g)
    _muon_check(g, _muon_grad(shape, 2, F32, 5e-3))


@pytest.mark.parametrize("kw", [dict(nesterov=False), dict(beta=0.0), dict(beta=-0.5), dict(steps=1), dict(steps=2),
                                dict(steps=7), dict(eps=1e-3), dict(steps=3, coeffs=[(4.0, -7.0, 4.0), (3.0, -3.2, 1.2),
                                                                                    (1.875, -1.25, 0.375)])])
def test_muon_update_arguments(kw):
    for shape in ((96, 160), (160, 96)):
        _muon_check(_muon_grad(shape, 3, BF), _muon_grad(shape, 4, F32), **kw)


@pytest.mark.parametrize("std", [1e-36, 1e-20, 1e-7, 1e6, 1e18, 1e35])
def test_muon_update_of_any_size(std):
    """The norm neither vanishes nor overflows (eps below the smallest norm)."""
    _muon_check(_muon_grad((70, 64), 5, F32, std), eps=1e-30)


@pytest.mark.parametrize("shape", [(20, 300, 328), (9, 700, 520), (12, 704, 1304), (16, 1300, 704), (1, 1999, 2304),
                                   (3, 1536, 1544), (2, 40, 8200), (2, 4100, 40), (200, 24, 24)])
def test_muon_update_many_tiles(shape):
    """Several tiles a side (of one block, and of pairs), ragged last ones, more
    tiles than teams; against the formula in 64 bits on the GPU."""
    g, m = _muon_grad(shape, 21, BF).cuda(), _muon_grad(shape, 22, F32, 3e-3).cuda()
    m1, m2 = m.clone(), m.clone()
    o, o2 = da.muon_update(g, momentum=m1), da.muon_update(g, momentum=m2)
    _done()
    assert torch.equal(o, o2) and torch.equal(m1, m2)
    w = 0.95 * m.double() + g.double()
    assert float((m1 - w).abs().max()) <= 2.0 ** -21 * float(w.abs().max())
    u = g.double() + 0.95 * w
    x = u / (torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + 1e-7)
    tall = shape[1] > shape[2]
    x = x.mT if tall else x
    held = lambda v, s: (v * s).half().double() / s
    y = held(x, 4096.0)
    for k in range(5):
        gram = x @ x.mT
        x = 3.4445 * x + (-4.7750 * gram + 2.0315 * gram @ gram) @ x
        gram = held(y @ y.mT, 4096.0)
        eye = torch.eye(gram.shape[-1], dtype=torch.float64, device="cuda")
        y = held(3.4445 * eye - 4.7750 * gram + 2.0315 * gram @ gram, 1024.0) @ y
        y = held(y, 4096.0) if k < 4 else y
    # As in _muon_check, matrix by matrix.
    got, want, near = o.double(), (x.mT if tall else x), (y.mT if tall else y)
    norm = torch.linalg.vector_norm(want, dim=(1, 2))
    off = torch.linalg.vector_norm(got - want, dim=(1, 2))
    tol = 2 * torch.linalg.vector_norm(near - want, dim=(1, 2)) + 2.0 ** -8 * norm
    assert bool((off <= tol).all()), (off / norm).max()


def test_muon_update_zero_and_bad_matrices():
    g = _muon_grad((4, 64, 72), 6, F32)
    good = da.muon_update(g.cuda())
    g[1] = 0
    g[2, 5, 7] = NAN
    g[3, 0, 0] = INF
    o = da.muon_update(g.cuda())
    _done()
    assert torch.equal(o[0], good[0]) and (o[1] == 0).all() and o[2].isnan().all() and o[3].isnan().all()


def test_muon_update_uneven_spectrum():
    """A few directions with most of the norm: the others are known to 2^-11 of those."""
    g = _gen(7)
    a = torch.randn((200, 4), generator=g) @ torch.randn((4, 304), generator=g) + 0.05 * torch.randn((200, 304), generator=g)
    _muon_check(a)
    _muon_check(a.t().contiguous()[:, :200])


def test_muon_update_outputs_and_workspace():
    g = _muon_grad((2, 130, 64), 8, BF).cuda()
    m = _muon_grad((2, 130, 64), 9, F32).cuda()
    m1, m2 = m.clone(), m.clone()
    want = da.muon_update(g, momentum=m1)
    n = g.numel()
    buf = torch.full((n + 64,), 7.0, dtype=BF, device="cuda")
    ws = torch.full((da.muon_update_workspace_bytes(2, 130, 64),), 255, dtype=torch.uint8, device="cuda")
    o = da.muon_update(g, momentum=m2, out=buf[32:32 + n].view_as(g), workspace=ws)
    _done()
    assert torch.equal(o, want) and torch.equal(m1, m2)
    assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()
    with pytest.raises(da.DetAttnError, match="workspace"):
        da.muon_update(g, workspace=ws[:-1])
    with pytest.raises(TypeError):
        da.muon_update(g.half())
    with pytest.raises(TypeError):
        da.muon_update(g, momentum=m.to(BF))
    with pytest.raises(ValueError, match="coeffs"):
        da.muon_update(g, coeffs=[(1, 1, 1)])
    with pytest.raises(da.DetAttnError):
        da.muon_update(g[..., :60].contiguous())
    assert da.muon_update(g[:0]).shape == (0, 130, 64)


# ------------------------------------------------------------ alignment and large offsets
def test_outputs_and_workspaces_on_16_bytes():
    """Rows are stored 32 bytes at a time where outputs begin so, and workspaces
    begin anywhere on 16 bytes."""
    def shifted(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
        start = 16 // buf.element_size()
        return buf, buf[start:start + n].view(shape)

    def workspace(n):
        return torch.full((n + 16,), 255, dtype=torch.uint8, device="cuda")[16:]
    x, w, t = (a.cuda() for a in _ce_inputs(300, 64, 777, seed=41))
    loss, lse = da.linear_ce_fwd(x, w, t, workspace=workspace(da.linear_ce_fwd_workspace_bytes(300, 777, 64)))
    g = torch.full((300,), 0.01, device="cuda")
    want = da.linear_ce_bwd(x, w, t, lse, g)
    bufs, outs = zip(*(shifted(s, BF) for s in ((300, 64), (777, 64))))
    da.linear_ce_bwd(x, w, t, lse, g, dx=outs[0], dw=outs[1],
                     workspace=workspace(da.linear_ce_bwd_workspace_bytes(300, 777, 64)))
    m = _muon_grad((3, 160, 320), 42, BF).cuda()
    bo, o = shifted((3, 160, 320), BF)
    da.muon_update(m, out=o, workspace=workspace(da.muon_update_workspace_bytes(3, 160, 320)))
    _done()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert torch.equal(o, da.muon_update(m))
    for b, v in zip((*bufs, bo), (*outs, o)):
        assert (b[:8] == 7).all() and (b[8 + v.numel():] == 7).all()


def test_rope_past_2_31_elements():
    T = 440000
    q = torch.empty((1, T, 40, 128), dtype=BF, device="cuda")
    q[0, -3:] = torch.randn((3, 40, 128), generator=_gen(43)).to(BF).cuda()
    f, _ = da.rope_freqs(128)
    y, _ = da.rope_fwd(q, None, f, q_out=q)
    last = _f(q[0, -3:].clone())
    x = torch.randn((3, 40, 128), generator=_gen(43)).to(BF)
    _done()
    want = os_.rope(_f(x), np.arange(T - 3, T), _f(f))
    assert (np.abs(last - want) <= _rope_tol(_f(x), want, 1.0, BF)).all()


def test_linear_ce_past_2_31_elements():
    N, d, V = 1400100, 1536, 300
    x = torch.zeros((N, d), dtype=BF, device="cuda")
    tail, w, t = (a.cuda() for a in _ce_inputs(500, d, V, seed=44))
    x[-500:] = tail
    targets = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    targets[-500:] = t
    g = torch.full((N,), 1.0 / 256, device="cuda")
    loss, lse = da.linear_ce_fwd(x, w, targets)
    dx, dw = da.linear_ce_bwd(x, w, targets, lse, g)
    _done()
    ref_loss, ref_lse = da.linear_ce_fwd(tail, w, t)
    ref_dx, ref_dw = da.linear_ce_bwd(tail, w, t, ref_lse, g[:500])
    assert float((loss[-500:] - ref_loss).abs().max()) <= 1e-5 and not loss[:-500].any()
    assert float((lse[:-500] - float(np.log(V))).abs().max()) <= 1e-5
    for a, b in ((dx[-500:], ref_dx), (dw, ref_dw)):
        assert float((a.double() - b.double()).norm() / b.double().norm()) <= 2.0 ** -8
    assert not dx[:-500].any()


def test_muon_update_past_2_31_elements():
    batch, n = 520, 2048
    g = torch.zeros((batch, n, n), dtype=BF, device="cuda")
    g[-1] = _muon_grad((n, n), 45, BF).cuda()
    o = da.muon_update(g)
    want = da.muon_update(g[-1:].clone())
    _done()
    assert not o[:-1].any()
    # (The tiles of one matrix alone may be other ones: equal but for the roundings' order.)
    assert float((o[-1].double() - want[0].double()).norm() / want[0].double().norm()) <= 2.0 ** -8


# ------------------------------------------------------------ together
def _step(s):
    """One training step of a model of one attention layer with these ends."""
    q, k = da.rope_fwd(s["qkv"][:, :, :4], s["qkv"][:, :, 4:6], s["f"])
    v = s["qkv"][:, :, 6:].contiguous()
    o, lse_a = da.attn_fwd(q, k, v)
    x = o.view(2, 128, 256)
    loss, lse = da.linear_ce_fwd(x, s["w"], s["t"])
    dx, dw = da.linear_ce_bwd(x, s["w"], s["t"], lse, s["g"])
    dq, dk, dv = da.attn_bwd(q, k, v, o, lse_a, dx.view_as(o))
    dq, dk = da.rope_bwd(dq, dk, s["f"])
    dqkv = torch.cat([dq, dk, dv], dim=2).view(256, 512)
    up = da.muon_update(dqkv, momentum=s["m"])
    return loss, dw, dqkv, up


def _step_state(seed=0):
    g = _gen(seed)
    return {"qkv": torch.randn((2, 128, 8, 64), generator=g).to(BF).cuda(), "f": da.rope_freqs(64)[0],
            "w": (0.05 * torch.randn((1000, 256), generator=g)).to(BF).cuda(),
            "t": torch.randint(-1, 1000, (2, 128), generator=g, dtype=torch.int32).cuda(),
            "g": torch.full((2, 128), 1.0 / 256, device="cuda"), "m": torch.zeros((256, 512), device="cuda")}


def test_step_together_against_the_oracle():
    import oracle
    s = _step_state()
    loss, dw, dqkv, up = _step(s)
    _done()
    qkv, f = _f(s["qkv"]), _f(s["f"])
    pos = np.broadcast_to(np.arange(128), (2, 128))
    q, k, v = os_.rope(qkv[:, :, :4], pos, f), os_.rope(qkv[:, :, 4:6], pos, f), qkv[:, :, 6:].copy()
    o, lse = oracle.attn_fwd(q, k, v, 0.125, True)
    t, w, g = s["t"].cpu().numpy().reshape(-1), _f(s["w"]), _f(s["g"]).reshape(-1)
    want, _, _ = os_.linear_ce(o.reshape(256, 256), w, t)
    # q, k, o are rounded to bf16 on the way (2^-8 each); tolerances as for the attention alone.
    assert np.linalg.norm(_f(loss).reshape(-1) - want) <= 1e-2 * np.linalg.norm(want)
    dx, edw, _, _ = os_.linear_ce_grad(o.reshape(256, 256), w, t, g)
    assert np.linalg.norm(_f(dw) - edw) <= 2e-2 * np.linalg.norm(edw)
    dq, dk, dv, _, _ = oracle.attn_bwd(q, k, v, np.ascontiguousarray(dx.reshape(o.shape)), 0.125, True)
    dq, dk = os_.rope(dq, pos, f, back=True), os_.rope(dk, pos, f, back=True)
    e = np.concatenate([dq, dk, dv], axis=2).reshape(256, 512)
    assert np.linalg.norm(_f(dqkv) - e) <= 2e-2 * np.linalg.norm(e)
    # The update of the gradient that was formed here.
    eu, em = os_.muon(_f(dqkv), np.zeros((256, 512)))
    held, _ = os_.muon(_f(dqkv), np.zeros((256, 512)), rounding=os_.to_fp16)
    assert np.linalg.norm(_f(up) - eu) <= 2 * np.linalg.norm(held - eu) + 2.0 ** -8 * np.linalg.norm(eu)


def test_step_repeats_bit_for_bit():
    runs = []
    for _ in range(3):
        s = _step_state()
        runs.append([t.clone() for t in _step(s)] + [s["m"]])
    _done()
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert torch.equal(a, b)


def test_step_captured_and_replayed():
    s, c = _step_state(1), _step_state(1)
    want = [[t.clone() for t in _step(s)] + [s["m"].clone()] for _ in range(2)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        _step(c)                       # warm up
        c["m"].zero_()
        graph = torch.cuda.CUDAGraph()
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            out = _step(c)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(w, list(out) + [c["m"]]):
            assert torch.equal(a, b)
    da.check_status()


def test_step_on_two_streams_at_once():
    a, b = _step_state(2), _step_state(3)
    want = [[t.clone() for t in _step(s)] for s in (a, b)]
    for s in (a, b):
        s["m"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, (s, st) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(st):
                s["m"].zero_()
                got[i] = _step(s)
    torch.cuda.synchronize()
    da.check_status()
    for w, g in zip(want, got):
        for x, y in zip(w, g):
            assert torch.equal(x, y)


def test_updates_on_two_streams_at_once():
    """Two launches whose blocks wait on one another share the GPU, and one the GPU with
    other work."""
    a, b = (_muon_grad(s, 30, BF).cuda() for s in ((6, 512, 640), (1, 900, 1000)))
    x, w, t = (v.cuda() for v in _ce_inputs(512, 256, 5000, seed=31))
    want = [da.muon_update(a), da.muon_update(b), *da.linear_ce_fwd(x, w, t)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [None] * 4
    for _ in range(10):
        with torch.cuda.stream(streams[0]):
            got[0] = da.muon_update(a)
        with torch.cuda.stream(streams[1]):
            got[1] = da.muon_update(b)
        with torch.cuda.stream(streams[2]):
            got[2], got[3] = da.linear_ce_fwd(x, w, t)
    torch.cuda.synchronize()
    da.check_status()
    for p, q in zip(want, got):
        assert torch.equal(p, q)


def test_two_updates_in_one_graph_share_a_workspace():
    g = _muon_grad((2, 300, 520), 32, BF).cuda()
    m1, m2 = (torch.zeros((2, 300, 520), device="cuda") for _ in range(2))
    ws = torch.empty((da.muon_update_workspace_bytes(2, 300, 520),), dtype=torch.uint8, device="cuda")
    o1, o2 = torch.empty_like(g), torch.empty_like(g)
    want = da.muon_update(g, momentum=m1, workspace=ws)
    want2 = da.muon_update(2 * g, momentum=m2, workspace=ws)
    torch.cuda.synchronize()
    g2 = 2 * g
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        m1.zero_(), m2.zero_()
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            m1.zero_(), m2.zero_()
            da.muon_update(g, momentum=m1, out=o1, workspace=ws)
            da.muon_update(g2, momentum=m2, out=o2, workspace=ws)
    for _ in range(3):
        o1.zero_(), o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want) and torch.equal(o2, want2)
    da.check_status()


def test_step_waits_that_run_out_are_named():
    da.selftest_wait_timeout(2_000_000)
    torch.cuda.synchronize()
    with pytest.raises(da.DetAttnError, match="linear_ce 1, muon_update 1"):
        da.check_status()
    da.check_status()
