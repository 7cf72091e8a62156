"""GPU parity of the block norms, 8-bit checkpoints, the weight gradient taken
from one and the gated unit against oracle.block in fp64.

Tolerances, from the arithmetic.  Everything between the loads and the stores
is fp32 (u = 2^-24); a bf16 store adds half a step, 2^-8 relative.

* An element of a row result is a handful of products around one sum over the
  row.  A lane adds at most 32 terms one after the other, then five shuffles
  and at most eleven warps; with the factors around it (and __expf's few units
  where the gate is a sigmoid) fewer than 64 roundings, each at most u times
  the magnitudes involved: |error| <= 64 u mag (+ 2^-8 |value| in bf16), mag
  being the sum of the magnitudes that the oracle returns beside the value.
* A column sum over N rows adds terms each of which is off by 64 u of its
  magnitude, in at most N + 200 additions: |error| <= (N + 264) u sum |terms|.
* A checkpoint made from a bf16 tensor is exact.  One made from normed values
  rounds a number that is off by 64 u: at most half a step and a thousandth
  (64 u 127 < 5e-4), with the exponent of a maximum within 1e-5 of the bound.
* The weight gradient's products are exact in fp32, and the tensor core adds
  rows of them in fp32: |error| <= (rows + 4) 2^-23 sum |terms| (2^-23: its
  additions may round towards zero), and rel-L2 <= 1e-5.
* The gated unit's __expf and __fdividef are within 2^-20 of their values for
  the arguments here, far below half a bf16 step: 2^-8 |value| + 2^-18 mag.
"""
import numpy as np
import pytest
import torch

import deterministic_attention_gb300 as da
from helpers import rel_l2, sha256, to_np
from oracle import block as ob

U = 2.0 ** -24
EPS = 1e-6


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _acts(g, rows, d, std=1.0):
    """bf16 activations with a few wide channels."""
    x = torch.randn((rows, d), generator=g) * std
    return (x * torch.where(torch.rand((d,), generator=g) < 0.03, 12.0, 1.0)).to(torch.bfloat16)


def _within(name, got, ref, mag, k, half):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    bound = half * np.abs(ref) + k * U * np.asarray(mag, np.float64) + 1e-38
    err = np.abs(got - ref)
    bad = err > bound
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} past the bound, worst "
                           f"{float((err / bound).max()):.3g} times it")


def _half(t):
    return 2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0


def _check_kept(name, c, ref, exact=False):
    """An 8-bit checkpoint of the values ref."""
    q, e = c.q.cpu().numpy(), c.e.cpu().numpy()
    if exact:
        rq, re = ob.act8(ref)
        assert np.array_equal(e, re) and np.array_equal(q, rq), name
    k = np.repeat(e.astype(np.int64) - 127, 32, axis=1)
    step = np.ldexp(1.0, k)
    big = np.abs(ref).reshape(ref.shape[0], -1, 32).max(-1)
    unit = step.reshape(ref.shape[0], -1, 32)[..., 0]
    assert np.all(big <= 127.0 * unit * (1 + 1e-5)), name
    assert np.all((big > 63.5 * unit * (1 - 1e-5)) | (e == 1)), name
    assert np.all(np.abs(ob.act8_values(q, e) - ref) <= 0.501 * step), name
    assert torch.equal(da.act8_unpack(c).cpu(), torch.from_numpy(ob.act8_values(q, e)).to(torch.bfloat16))


# ------------------------------------------------------------ checkpoints
@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(1, 32), (3, 64), (5, 4096), (129, 96), (1000, 1184), (2, 1 << 20)])
def test_act8_round_trip_is_exact(rows, d):
    x = _acts(_gen(rows + d), rows, d)
    x.view(-1)[::7] *= 2.0 ** -130   # groups of small numbers, subnormal ones among them
    x[0, :32] = 0
    c = da.act8_pack(x.cuda())
    _check_kept("pack", c, to_np(x), exact=True)


@pytest.mark.gpu
def test_act8_extremes():
    x = torch.zeros((6, 64), dtype=torch.bfloat16)
    x[0, 3], x[0, 40] = float("inf"), float("nan")
    x[1, 0], x[1, 33] = 3.3895e38, -3.3895e38   # the largest bf16 numbers
    x[2, :] = -0.0
    x[3, :32], x[3, 32:] = 127.0, 127.5
    x[4, 7] = torch.finfo(torch.bfloat16).tiny
    x[5, 31] = 9.2e-41                          # subnormal
    c = da.act8_pack(x.cuda())
    q, e = ob.act8(to_np(x))
    assert np.array_equal(c.e.cpu().numpy(), e) and np.array_equal(c.q.cpu().numpy(), q)
    back = da.act8_unpack(c).cpu()
    assert back[0].isnan().all() and back[1:].isfinite().all()
    assert np.array_equal(to_np(back[1:]), ob.act8_values(q, e)[1:])


@pytest.mark.gpu
def test_act8_empty():
    c = da.act8_pack(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert c.q.shape == (0, 64) and c.e.shape == (0, 2) and da.act8_unpack(c).shape == (0, 64)


# ------------------------------------------------------------ weight gradient
@pytest.mark.gpu
@pytest.mark.parametrize("rows,d,n", [
    (1, 32, 8), (63, 64, 256), (64, 128, 264), (65, 160, 8), (500, 96, 1000), (1777, 1184, 504),
    (4096, 768, 1280),       # every tile cut
    (192, 19 * 256, 4 * 256),  # exactly one whole tile for each pair of blocks, nothing cut
    (2500, 2496, 2200),      # whole tiles and cut ones, ragged both ways
    (200, 2432, 5000),       # a pair walks several whole tiles
    (2600, 4864, 1024),      # a whole tile takes its tokens in three runs
])
@pytest.mark.parametrize("scaled", [False, True])
def test_wgrad_matches_product(rows, d, n, scaled):
    g = _gen(rows + d + n)
    x, dy = _acts(g, rows, d), (0.1 * torch.randn((rows, n), generator=g)).to(torch.bfloat16)
    w = torch.randn((d,), generator=g) + 1.0
    q, e = ob.act8(to_np(x))
    vals = ob.act8_values(q, e)
    c = da.Act8(torch.from_numpy(q).cuda(), torch.from_numpy(e).cuda())
    k = to_np(w)[:, None] if scaled else 1.0
    ref, mag = k * (vals.T @ to_np(dy)), np.abs(k) * (np.abs(vals).T @ np.abs(to_np(dy)))
    dw = torch.full((d, n), float("nan"), device="cuda")
    ws = torch.full((max(16, da.act8_wgrad_workspace_bytes(rows, d, n)),), 255, dtype=torch.uint8,
                    device="cuda")
    da.act8_wgrad(c, dy.cuda(), row_scale=w.cuda() if scaled else None, dw=dw, workspace=ws)
    torch.cuda.synchronize()
    da.check_status()
    _within("dw", to_np(dw), ref, mag, 2 * (rows + 4), 0.0)
    assert rel_l2(to_np(dw), ref) <= 1e-5
    again = da.act8_wgrad(c, dy.cuda(), row_scale=w.cuda() if scaled else None)
    assert torch.equal(again, dw)


@pytest.mark.gpu
def test_wgrad_plan_cases_are_what_they_say():
    """The shapes above reach whole tiles only, cut tiles only, and both."""
    assert da.act8_wgrad_workspace_bytes(192, 19 * 256, 4 * 256) == 0
    assert da.act8_wgrad_workspace_bytes(4096, 768, 1280) == 15 * 5 * 256 * 256 * 4
    assert da.act8_wgrad_workspace_bytes(2500, 2496, 2200) == 14 * 5 * 256 * 256 * 4


@pytest.mark.gpu
def test_wgrad_no_rows_gives_zeros():
    c = da.Act8(torch.empty((0, 64), dtype=torch.int8, device="cuda"),
                torch.empty((0, 2), dtype=torch.uint8, device="cuda"))
    dw = torch.full((64, 16), float("nan"), device="cuda")
    da.act8_wgrad(c, torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"), dw=dw)
    assert torch.equal(dw, torch.zeros_like(dw))


@pytest.mark.gpu
def test_wgrad_marked_group_reaches_its_own_rows_only():
    """A group that held an infinity reads as NaN: dw's 32 rows of that group
    are NaN, every other row is as without it."""
    g = _gen(9)
    x, dy = _acts(g, 100, 256), torch.randn((100, 64), generator=g).to(torch.bfloat16).cuda()
    clean = da.act8_wgrad(da.act8_pack(x.cuda()), dy)
    x[17, 70] = float("inf")
    dw = da.act8_wgrad(da.act8_pack(x.cuda()), dy)
    assert dw[64:96].isnan().all()
    assert torch.equal(dw[:64], clean[:64]) and torch.equal(dw[96:], clean[96:])


# ------------------------------------------------------------ gated unit
@pytest.mark.gpu
@pytest.mark.parametrize("rows,f", [(1, 8), (3, 40), (7, 32), (130, 1000), (257, 2048)])
def test_swiglu_matches_oracle(rows, f):
    g = _gen(rows * f)
    u, dh = _acts(g, rows, 2 * f), torch.randn((rows, f), generator=g).to(torch.bfloat16)
    a, b = np.split(to_np(u), 2, axis=-1)
    s = ob.sigmoid(a)
    ref_h = ob.swiglu(to_np(u))
    _within("h", to_np(da.swiglu_fwd(u.cuda())), ref_h, np.abs(ref_h), 64, 2.0 ** -8)
    gmag = np.abs(to_np(dh))
    mag = np.concatenate([gmag * np.abs(b) * s * (1 + np.abs(a) * (1 - s)), gmag * np.abs(a) * s], -1)
    du, h = da.swiglu_bwd(dh.cuda(), u.cuda(), with_h=True)
    _within("du", to_np(du), ob.swiglu_grad(to_np(dh), to_np(u)), mag, 64, 2.0 ** -8)
    _within("h again", to_np(h), ref_h, np.abs(ref_h), 64, 2.0 ** -8)
    assert torch.equal(da.swiglu_bwd(dh.cuda(), u.cuda()), du)
    if f % 32:
        return
    h8, c = da.swiglu_fwd(u.cuda(), keep8=True)
    assert torch.equal(h8, da.swiglu_fwd(u.cuda()))
    _check_kept("u", c, to_np(u), exact=True)
    v = ob.act8_values(*ob.act8(to_np(u)))
    a, b = np.split(v, 2, axis=-1)
    s = ob.sigmoid(a)
    mag = np.concatenate([gmag * np.abs(b) * s * (1 + np.abs(a) * (1 - s)), gmag * np.abs(a) * s], -1)
    du, h = da.swiglu_bwd(dh.cuda(), c, with_h=True)
    _within("du from 8", to_np(du), ob.swiglu_grad(to_np(dh), v), mag, 64, 2.0 ** -8)
    _within("h from 8", to_np(h), ob.swiglu(v), np.abs(ob.swiglu(v)), 64, 2.0 ** -8)


@pytest.mark.gpu
def test_swiglu_large_arguments():
    """Far arguments: sigma goes to 0 or 1 without NaN while a is finite."""
    u = torch.tensor([[100.0, -100.0, 3e4, -3e4, 0.0, -0.0, 88.0, -88.0] + [1.0] * 8]).to(torch.bfloat16)
    dh = torch.ones((1, 8), dtype=torch.bfloat16)
    du, h = da.swiglu_bwd(dh.cuda(), u.cuda(), with_h=True)
    ref = ob.swiglu(to_np(u))
    assert np.abs(to_np(h) - ref).max() <= 2.0 ** -8 * np.abs(ref).max()
    assert np.all(np.abs(to_np(h) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-30)
    assert np.all(np.abs(to_np(du) - ob.swiglu_grad(to_np(dh), to_np(u))) <=
                  2.0 ** -8 * np.abs(ob.swiglu_grad(to_np(dh), to_np(u))) + 1e-30)


@pytest.mark.gpu
def test_swiglu_empty():
    u = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h, c = da.swiglu_fwd(u, keep8=True)
    assert h.shape == (0, 32) and da.swiglu_bwd(h, c).shape == (0, 64)


# ------------------------------------------------------------ block norms
def _norm_inputs(rows, d, gate, post, pre, stream, seed, block=True):
    g = _gen(seed)
    dt = torch.float32 if stream == "fp32" else torch.bfloat16
    i = {"x": _acts(g, rows, d).to(dt), "y": _acts(g, rows, d, 0.5) if block else None,
         "w_post": torch.randn((d,), generator=g) * 0.3 + 1 if post else None,
         "w_pre": torch.randn((d,), generator=g) * 0.3 + 1 if pre else None, "gate": None,
         "dx_out": torch.randn((rows, d), generator=g).to(dt),
         "dh": torch.randn((rows, d), generator=g).to(torch.bfloat16) if pre else None}
    if gate is not None:
        G, gdt = gate
        G = rows if G == "row" else G
        i["gate"] = torch.randn((G, d), generator=g).to(gdt)
    return i


def _cuda(i):
    return {k: (v.cuda() if v is not None else None) for k, v in i.items()}


def _np(t):
    return None if t is None else to_np(t)


F32, BF = torch.float32, torch.bfloat16
NORM_CASES = [
    # rows, d, gate (rows, type), sigmoid, norm after, norm before, stream
    (1, 32, None, False, True, True, "bf16"),
    (1, 8192, (1, F32), False, True, True, "fp32"),
    (2, 64, (2, BF), True, True, True, "bf16"),
    (5, 256, ("row", BF), True, True, True, "fp32"),
    (37, 768, (1, F32), False, True, True, "bf16"),
    (128, 768, None, False, False, True, "bf16"),
    (130, 800, (1, BF), True, False, True, "fp32"),
    (96, 1024, (3, F32), True, True, False, "bf16"),
    (64, 1056, ("row", F32), False, True, True, "bf16"),
    (1500, 512, (1, F32), False, True, True, "bf16"),
    (2000, 96, (250, F32), False, True, True, "bf16"),   # slices of a few rows
    (4000, 32, (2000, BF), False, True, True, "fp32"),   # more gate rows than blocks
    (333, 1536, (9, F32), True, True, True, "fp32"),
    (40, 4608, (2, F32), False, True, True, "fp32"),
    (24, 6400, ("row", BF), False, True, True, "fp32"),
    (2500, 2304, (1, F32), False, True, True, "bf16"),
    (50, 8192, (5, BF), False, False, True, "bf16"),
    (77, 3200, None, False, False, False, "fp32"),       # the residual add alone
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d,gate,sig,post,pre,stream", NORM_CASES)
@pytest.mark.parametrize("keep8", [False, True])
def test_block_norm_fwd_matches_oracle(rows, d, gate, sig, post, pre, stream, keep8):
    i = _norm_inputs(rows, d, gate, post, pre, stream, rows + d)
    c = _cuda(i)
    r, s = 0.9, 0.6
    x_out, h, kept = da.block_norm_fwd(c["x"], c["y"], gate=c["gate"], w_post=c["w_post"],
                                       w_pre=c["w_pre"], res_scale=r, block_scale=s, eps=EPS,
                                       gate_sigmoid=sig, keep8=keep8)
    torch.cuda.synchronize()
    o = ob.norm_fwd(_np(i["x"]), _np(i["y"]), _np(i["gate"]), _np(i["w_post"]), _np(i["w_pre"]), r,
                    s, EPS, sig)
    xm = np.abs(r * to_np(i["x"])) + np.abs(o["x"] - r * to_np(i["x"]))
    assert x_out.dtype == i["x"].dtype
    _within("x'", to_np(x_out), o["x"], xm, 64, _half(x_out))
    if post:
        _within("rstd_post", to_np(kept.rstd_post), o["rstd_post"], o["rstd_post"], 64, 0.0)
    if pre:
        # The row's mean square is off by 64 u of the sum of mag^2.
        stat = np.sqrt((xm ** 2).sum(-1) / np.maximum((o["x"] ** 2).sum(-1), 1e-300))
        _within("rstd_pre", to_np(kept.rstd_pre), o["rstd_pre"], o["rstd_pre"] * stat, 64, 0.0)
        _within("h", to_np(h), o["h"],
                np.abs(to_np(i["w_pre"])) * o["rstd_pre"][:, None] * (xm + np.abs(o["x"]) * stat[:, None]),
                64, 2.0 ** -8)
    if keep8:
        assert kept.x is None and kept.y is None
        _check_kept("yhat", kept.yhat8, o["yhat"], exact=not post)
        if pre:
            _check_kept("xhat", kept.xhat8, o["xhat"])
    else:
        assert kept.x is x_out and kept.y is c["y"]


def _bwd_refs(i, kept, r, s, sig, block=True):
    xhat = yhat = None
    if kept.xhat8 is not None:
        xhat = ob.act8_values(kept.xhat8.q.cpu().numpy(), kept.xhat8.e.cpu().numpy())
    elif i["w_pre"] is not None:
        xhat = to_np(kept.x.cpu()) * to_np(kept.rstd_pre.cpu())[:, None]
    if kept.yhat8 is not None:
        yhat = ob.act8_values(kept.yhat8.q.cpu().numpy(), kept.yhat8.e.cpu().numpy())
    elif block:
        yhat = to_np(kept.y.cpu())
        if i["w_post"] is not None:
            yhat = yhat * to_np(kept.rstd_post.cpu())[:, None]
    dx_out = i["dx_out"] if i["dx_out"] is not None else torch.zeros_like(i["x"])
    rp = None if kept.rstd_pre is None else to_np(kept.rstd_pre.cpu())
    ro = None if kept.rstd_post is None else to_np(kept.rstd_post.cpu())
    return ob.norm_bwd(to_np(dx_out), _np(i["dh"]), xhat, yhat, rp, ro, _np(i["gate"]),
                       _np(i["w_post"]), _np(i["w_pre"]), r, s, sig, block)


def _check_bwd(got, o, rows):
    for name, v in got._asdict().items():
        assert (v is None) == (name not in o), name
        if v is None:
            continue
        k = 64 if name in ("dx", "dy") else rows + 264
        _within(name, to_np(v), o[name].reshape(v.shape), o["|%s|" % name].reshape(v.shape), k, _half(v))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d,gate,sig,post,pre,stream", NORM_CASES)
@pytest.mark.parametrize("keep8", [False, True])
def test_block_norm_bwd_matches_oracle(rows, d, gate, sig, post, pre, stream, keep8):
    i = _norm_inputs(rows, d, gate, post, pre, stream, rows + 3 * d)
    c = _cuda(i)
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], res_scale=0.9, block_scale=0.6,
              gate_sigmoid=sig)
    _, _, kept = da.block_norm_fwd(c["x"], c["y"], eps=EPS, keep8=keep8, **kw)
    G = 1 if c["gate"] is None else c["gate"].shape[0]
    outs = []
    for fill in (255, 0):
        ws = torch.full((da.block_norm_bwd_workspace_bytes(rows, d, G),), fill, dtype=torch.uint8,
                        device="cuda")
        outs.append(da.block_norm_bwd(c["dx_out"], c["dh"], kept, workspace=ws, **kw))
    torch.cuda.synchronize()
    da.check_status()
    _check_bwd(outs[0], _bwd_refs(i, kept, 0.9, 0.6, sig), rows)
    for a, b in zip(*outs):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d,stream", [(1, 8, "bf16"), (13, 1000, "bf16"), (600, 776, "fp32"),
                                           (9, 8192, "fp32")])
def test_block_norm_without_block(rows, d, stream):
    """The norm before the first block: no y, x' is x."""
    i = _norm_inputs(rows, d, None, False, True, stream, 7, block=False)
    c = _cuda(i)
    x_out, h, kept = da.block_norm_fwd(c["x"], w_pre=c["w_pre"], eps=EPS)
    assert x_out is c["x"]
    o = ob.norm_fwd(to_np(i["x"]), w_pre=to_np(i["w_pre"]), eps=EPS)
    _within("h", to_np(h), o["h"], np.abs(o["h"]), 64, 2.0 ** -8)
    got = da.block_norm_bwd(c["dx_out"], c["dh"], kept, w_pre=c["w_pre"])
    assert got.dy is None
    _check_bwd(got, _bwd_refs(i, kept, 1.0, 1.0, False, block=False), rows)
    i["dx_out"] = None  # nothing comes back along the stream
    got = da.block_norm_bwd(None, c["dh"], kept, w_pre=c["w_pre"])
    assert got.dx.dtype == i["x"].dtype
    _check_bwd(got, _bwd_refs(i, kept, 1.0, 1.0, False, block=False), rows)


@pytest.mark.gpu
def test_block_norm_no_rows():
    d = 64
    w = torch.ones(d, device="cuda")
    x = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    gate = torch.ones((1, d), device="cuda")
    _, h, kept = da.block_norm_fwd(x, x, gate=gate, w_post=w, w_pre=w)
    assert h.shape == (0, d)
    got = da.block_norm_bwd(x, h, kept, gate=gate, w_post=w, w_pre=w)
    for t in (got.dw_pre, got.dw_post, got.dgate):
        assert torch.equal(t, torch.zeros_like(t))


@pytest.mark.gpu
def test_block_norm_in_place_and_3d():
    """x' may overwrite x and dx may overwrite dx_out; a [B, T, d] stream with a
    [B, d] gate is the [B T, d] one with its gate rows."""
    B, T, d = 4, 50, 768
    i = _norm_inputs(B * T, d, (B, F32), True, True, "bf16", 11)
    c = _cuda(i)
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], res_scale=0.5)
    x_out, h, kept = da.block_norm_fwd(c["x"], c["y"], **kw)
    ref = da.block_norm_bwd(c["dx_out"], c["dh"], kept, **kw)
    x3, y3 = c["x"].clone().view(B, T, d), c["y"].view(B, T, d)
    x_out3, h3, kept3 = da.block_norm_fwd(x3, y3, x_out=x3, **kw)
    assert x_out3 is x3 and torch.equal(x3.view(-1, d), x_out) and torch.equal(h3.view(-1, d), h)
    dx = c["dx_out"].clone().view(B, T, d)
    got = da.block_norm_bwd(dx, c["dh"].view(B, T, d), kept3, dx=dx, **kw)
    assert got.dx is dx
    for a, b in zip(got, ref):
        assert torch.equal(a.reshape(b.shape), b)


@pytest.mark.gpu
def test_block_norm_rows_do_not_touch_each_other():
    """A row of infinities or NaN spoils its own results (and the column sums),
    no other row's."""
    i = _norm_inputs(40, 768, ("row", BF), True, True, "bf16", 13)
    kw = {k: (i[k].cuda() if i[k] is not None else None) for k in ("gate", "w_post", "w_pre")}
    clean = da.block_norm_fwd(i["x"].cuda(), i["y"].cuda(), keep8=True, **kw)
    x, y = i["x"].clone(), i["y"].clone()
    x[5, 3], y[9, 700] = float("nan"), float("inf")
    got = da.block_norm_fwd(x.cuda(), y.cuda(), keep8=True, **kw)
    rest = [t for t in range(40) if t not in (5, 9)]
    for a, b in ((got[0], clean[0]), (got[1], clean[1]), (got[2].rstd_pre, clean[2].rstd_pre),
                 (got[2].xhat8.q, clean[2].xhat8.q), (got[2].yhat8.e, clean[2].yhat8.e)):
        assert torch.equal(a[rest], b[rest])
    assert got[1][5].isnan().all() and (got[2].xhat8.e[5] == 255).all()
    grads = da.block_norm_bwd(i["dx_out"].cuda(), i["dh"].cuda(), got[2], **kw)
    ref = da.block_norm_bwd(i["dx_out"].cuda(), i["dh"].cuda(), clean[2], **kw)
    for a, b in ((grads.dx, ref.dx), (grads.dy, ref.dy), (grads.dgate, ref.dgate)):
        assert torch.equal(a[rest], b[rest])
    assert grads.dx[5].isnan().all() and grads.dw_pre.isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_block_norm_rows_of_zeros_and_tiny_values(stream):
    """Padding rows: everything they give is zero, in their checkpoints too
    (1 / rms is then 1 / sqrt(eps)); groups far below 1 keep their values."""
    i = _norm_inputs(12, 256, (1, F32), True, True, stream, 43)
    i["x"][3:6], i["y"][3:6] = 0, 0
    i["x"][7, 64:128] = 2.0 ** -100
    i["y"][7, 64:128] = -(2.0 ** -120)
    i["x"][9], i["y"][9] = 2.0 ** -110, 2.0 ** -126
    c = _cuda(i)
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"])
    x_out, h, kept = da.block_norm_fwd(c["x"], c["y"], eps=EPS, keep8=True, **kw)
    o = ob.norm_fwd(_np(i["x"]), _np(i["y"]), _np(i["gate"]), _np(i["w_post"]), _np(i["w_pre"]), eps=EPS)
    _check_kept("yhat", kept.yhat8, o["yhat"])
    _check_kept("xhat", kept.xhat8, o["xhat"])
    for t in (x_out, h, kept.xhat8.q, kept.yhat8.q):
        assert not t[3:6].any()
    assert (kept.xhat8.e[3:6] == 1).all() and (kept.yhat8.e[3:6] == 1).all()
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"])
    _check_bwd(da.block_norm_bwd(c["dx_out"], c["dh"], kept, **kw), _bwd_refs(i, kept, 1.0, 1.0, False), 12)


@pytest.mark.gpu
def test_block_norm_smallest_eps():
    """1 / sqrt(eps) near the largest fp32 powers: a row of zeros stays zero."""
    x = torch.zeros((2, 64), dtype=BF, device="cuda")
    x[1] = 1.0
    _, h, kept = da.block_norm_fwd(x, w_pre=torch.ones(64, device="cuda"), eps=1e-44, keep8=True)
    assert not h[0].any() and not kept.xhat8.q[0].any() and (kept.xhat8.e[0] == 1).all()
    assert torch.equal(h[1].float(), torch.ones(64, device="cuda"))
    assert torch.equal(da.act8_unpack(kept.xhat8)[1], h[1])


# ------------------------------------------------------------ identity, streams, graphs
def _everything(i, dy):
    kw = dict(gate=i["gate"], w_post=i["w_post"], w_pre=i["w_pre"], res_scale=0.9, block_scale=0.6)
    x_out, h, kept = da.block_norm_fwd(i["x"], i["y"], keep8=True, **kw)
    got = da.block_norm_bwd(i["dx_out"], i["dh"], kept, **kw)
    dw = da.act8_wgrad(kept.xhat8, dy, row_scale=i["w_pre"])
    hh, u8 = da.swiglu_fwd(h, keep8=True)
    du, h2 = da.swiglu_bwd(hh, u8, with_h=True)
    return [x_out, h, *got, dw, hh, du, h2, da.act8_unpack(da.act8_pack(h))]


@pytest.mark.gpu
def test_twenty_runs_bit_identical():
    i = _cuda(_norm_inputs(1111, 1536, (1, F32), True, True, "bf16", 17))
    dy = torch.randn((1111, 776), generator=_gen(3)).to(BF).cuda()
    first = None
    for _ in range(20):
        d = [sha256(t) for t in _everything(i, dy)]
        first = first or d
        assert d == first
    da.check_status()


@pytest.mark.gpu
def test_side_stream_and_captured_graph_give_the_same_bits():
    i = _cuda(_norm_inputs(700, 768, (7, F32), True, True, "bf16", 19))
    dy = torch.randn((700, 264), generator=_gen(4)).to(BF).cuda()
    ref = _everything(i, dy)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        side = _everything(i, dy)
    st.synchronize()
    for a, b in zip(ref, side):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = _everything(i, dy)
    i["y"].mul_(2)          # new inputs, same addresses
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, _everything(i, dy)):
        assert torch.equal(a, b)
    da.check_status()


@pytest.mark.gpu
def test_outputs_stay_inside_their_buffers():
    """Guard bytes around every output of ragged calls stay as they were."""
    rows, d, n = 67, 1056, 136
    i = _cuda(_norm_inputs(rows, d, (1, F32), True, True, "bf16", 23))
    guarded = []

    def buf(shape, dtype):
        size = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        guarded.append((raw, size))
        return raw[256:256 + size].view(dtype).view(shape)

    kw = dict(gate=i["gate"], w_post=i["w_post"], w_pre=i["w_pre"])
    x_out, h, kept = da.block_norm_fwd(i["x"], i["y"], keep8=True, x_out=buf((rows, d), BF), **kw)
    ws = buf((da.block_norm_bwd_workspace_bytes(rows, d, 1),), torch.uint8)
    da.block_norm_bwd(i["dx_out"], i["dh"], kept, dx=buf((rows, d), BF), workspace=ws, **kw)
    c = da.act8_pack(h, out=da.Act8(buf((rows, d), torch.int8), buf((rows, d // 32), torch.uint8)))
    da.act8_unpack(c, out=buf((rows, d), BF))
    dy = torch.randn((rows, n), generator=_gen(5)).to(BF).cuda()
    da.act8_wgrad(c, dy, dw=buf((d, n), F32),
                  workspace=buf((max(16, da.act8_wgrad_workspace_bytes(rows, d, n)),), torch.uint8))
    u = i["x"][:, :64 * 16].contiguous()
    da.swiglu_bwd(da.swiglu_fwd(u, out=buf((rows, 512), BF)), u, du=buf((rows, 1024), BF))
    torch.cuda.synchronize()
    for raw, size in guarded:
        assert (raw[:256] == 0xA5).all() and (raw[256 + size:] == 0xA5).all()


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two calls of everything under way at the same time, each with its own
    outputs and workspaces, give what each gives alone."""
    a = _cuda(_norm_inputs(3000, 768, (1, F32), True, True, "bf16", 29))
    b = _cuda(_norm_inputs(2000, 1024, (4, F32), True, True, "fp32", 31))
    dya = torch.randn((3000, 512), generator=_gen(6)).to(BF).cuda()
    dyb = torch.randn((2000, 1032), generator=_gen(7)).to(BF).cuda()
    ref_a, ref_b = _everything(a, dya), _everything(b, dyb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(sa):
            outs.append((ref_a, _everything(a, dya)))
        with torch.cuda.stream(sb):
            outs.append((ref_b, _everything(b, dyb)))
    torch.cuda.synchronize()
    da.check_status()
    for ref, got in outs:
        for x, y in zip(ref, got):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_two_graphs_share_a_workspace():
    """Replayed one after the other, two graphs may use the same workspaces:
    nothing is carried over in them."""
    i = _cuda(_norm_inputs(900, 768, (1, F32), True, True, "bf16", 37))
    kw = dict(gate=i["gate"], w_post=i["w_post"], w_pre=i["w_pre"])
    _, _, kept = da.block_norm_fwd(i["x"], i["y"], keep8=True, **kw)
    dy = torch.randn((900, 384), generator=_gen(8)).to(BF).cuda()
    ws = torch.empty(da.block_norm_bwd_workspace_bytes(900, 768, 1), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(max(16, da.act8_wgrad_workspace_bytes(900, 768, 384)), dtype=torch.uint8, device="cuda")

    def run(dx_out):
        g = da.block_norm_bwd(dx_out, i["dh"], kept, workspace=ws, **kw)
        return [*g, da.act8_wgrad(kept.xhat8, dy, workspace=ws2)]

    d2 = i["dx_out"].flip(0).contiguous()
    refs = [run(i["dx_out"]), run(d2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in (i["dx_out"], d2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(d))
        graphs.append(g)
    for k in (0, 1, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    for ref, got in zip(refs, outs):
        for x, y in zip(ref, got):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: their last rows equal, bit for bit,
    the same rows on their own."""
    tail, d = 37, 2048
    rows = (1 << 20) + 5
    x = torch.zeros((rows, d), dtype=BF, device="cuda")
    x[-tail:] = torch.randn((tail, d), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF)
    end = x[-tail:].clone()
    c, ce = da.act8_pack(x), da.act8_pack(end)
    assert torch.equal(c.q[-tail:], ce.q) and torch.equal(c.e[-tail:], ce.e)
    assert torch.equal(da.act8_unpack(c)[-tail:], da.act8_unpack(ce))
    h, u8 = da.swiglu_fwd(x, keep8=True)
    he, _ = da.swiglu_fwd(end, keep8=True)
    assert torch.equal(h[-tail:], he) and torch.equal(u8.q[-tail:], ce.q) and torch.equal(u8.e[-tail:], ce.e)
    for u, ue in ((x, end), (c, ce)):
        assert torch.equal(da.swiglu_bwd(h, u)[-tail:], da.swiglu_bwd(he, ue))
    del h, he, u8, u
    w = torch.ones(d, device="cuda")
    for keep8 in (False, True):
        kw = dict(gate=w, w_post=w, w_pre=w)
        got = da.block_norm_fwd(x, x, keep8=keep8, **kw)
        ref = da.block_norm_fwd(end, end, keep8=keep8, **kw)
        for a, b in zip(got[:2], ref[:2]):
            assert torch.equal(a[-tail:], b)
        got = da.block_norm_bwd(x, x, got[2], **kw)
        ref = da.block_norm_bwd(end, end, ref[2], **kw)
        for a, b in zip(got[:2], ref[:2]):
            assert torch.equal(a[-tail:], b)
        # Rows of zeros add nothing; the sums' order differs between the two:
        # 37 terms and as many roundings of at most 2^-24 of the sum of magnitudes.
        for a, b in zip(got[2:], ref[2:]):
            assert (a - b).abs().max() <= 37 * 2.0 ** -23 * 37 * 25
        del got, ref
    # Whole numbers, so every order of summing gives the same bits.
    del x
    dy = torch.zeros((rows, 8), dtype=BF, device="cuda")
    dy[-tail:] = torch.randint(-4, 5, (tail, 8), device="cuda").to(BF)
    q = torch.zeros((rows, d), dtype=torch.int8, device="cuda")
    q[-tail:] = torch.randint(-127, 128, (tail, d), device="cuda").to(torch.int8)
    e = torch.full((rows, d // 32), 127, dtype=torch.uint8, device="cuda")
    assert torch.equal(da.act8_wgrad(da.Act8(q, e), dy), q[-tail:].double().T.matmul(dy[-tail:].double()).float())
    del q, e, dy, c
    q = torch.randint(-127, 128, (40, 1 << 16), device="cuda").to(torch.int8)
    dy = torch.randint(-4, 5, (40, (1 << 15) + 8), device="cuda").to(BF)
    e = torch.full((40, 1 << 11), 127, dtype=torch.uint8, device="cuda")
    dw = da.act8_wgrad(da.Act8(q, e), dy)
    assert torch.equal(dw[-300:, -300:], q[:, -300:].double().T.matmul(dy[:, -300:].double()).float())
    assert torch.equal(dw[:300, :300], q[:, :300].double().T.matmul(dy[:, :300].double()).float())


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit():
    x = torch.zeros((8, 64), dtype=BF, device="cuda")
    w, gate = torch.ones(64, device="cuda"), torch.ones((3, 64), device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        da.act8_pack(torch.zeros((8, 128), dtype=BF, device="cuda")[:, ::2])
    with pytest.raises(ValueError, match="multiple of 32"):
        da.act8_pack(torch.zeros((8, 40), dtype=BF, device="cuda"))
    with pytest.raises(TypeError):
        da.act8_pack(x.float())
    with pytest.raises(ValueError, match="divides"):
        da.block_norm_fwd(x, x, gate=gate, w_pre=w)
    with pytest.raises(ValueError, match="belong to"):
        da.block_norm_fwd(x, w_post=w, w_pre=w)
    with pytest.raises(TypeError):
        da.block_norm_fwd(x, w_pre=w.to(BF))
    with pytest.raises(TypeError):
        da.block_norm_fwd(x.half(), w_pre=w)
    with pytest.raises(da.DetAttnError):
        da.block_norm_fwd(x, w_pre=w, eps=0.0)
    with pytest.raises(da.DetAttnError):
        da.block_norm_fwd(x)                     # neither a block nor a norm
    with pytest.raises(da.DetAttnError):
        big = torch.zeros((1, 8200), dtype=BF, device="cuda")
        da.block_norm_fwd(big, w_pre=torch.ones(8200, device="cuda"))
    _, h, kept = da.block_norm_fwd(x, x, w_post=w, w_pre=w)
    with pytest.raises(ValueError, match="go together"):
        da.block_norm_bwd(x, None, kept, w_post=w, w_pre=w)
    with pytest.raises(TypeError):
        da.block_norm_bwd(x.float(), h, kept, w_post=w, w_pre=w)   # kept.x is bf16
    with pytest.raises(TypeError, match="kept.x"):                # without dx_out, kept.x says the type
        da.block_norm_bwd(None, h, kept._replace(x=x.half(), y=None), w_pre=w)
    with pytest.raises(ValueError, match="rows"):
        da.act8_wgrad(da.act8_pack(x), torch.zeros((7, 64), dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        da.swiglu_bwd(x, x)
    with pytest.raises(da.DetAttnError):
        da.act8_wgrad(da.act8_pack(x), torch.zeros((8, 12), dtype=BF, device="cuda"))


# ------------------------------------------------------------ together
def _split_heads(qkv, B, T, Hq, Hkv, D):
    q, k, v = torch.split(qkv.view(B, T, -1, D), [Hq, Hkv, Hkv], dim=2)
    return q.contiguous(), k.contiguous(), v.contiguous()


def _decoder_layer(t, B, T, Hq, Hkv, D):
    """One decoder layer's step as a training loop would run it: norm,
    projection, attention, projection, norm + gate + residual + norm, gated
    unit, norm + residual, and back, with every activation that the weight
    gradients need kept in 8 bits."""
    r, s, rows = 0.9, 0.7, B * T
    _, h1, k1 = da.block_norm_fwd(t["x"], w_pre=t["w1"], keep8=True)
    q, k, v = _split_heads(da.layer_gemm(h1, t["wqkv"]), B, T, Hq, Hkv, D)
    o, lse = da.attn_fwd(q, k, v)
    y = da.layer_gemm(o.view(rows, -1), t["wo"])
    kw = dict(gate=t["gate"], w_post=t["wp"], w_pre=t["w2"], res_scale=r, block_scale=s)
    x1, h2, k2 = da.block_norm_fwd(t["x"], y, keep8=True, **kw)
    hu, u8 = da.swiglu_fwd(da.layer_gemm(h2, t["wu"]), keep8=True)
    x2, _, k3 = da.block_norm_fwd(x1, da.layer_gemm(hu, t["wd"]), w_post=t["wp2"], keep8=True)

    b3 = da.block_norm_bwd(t["dx"], None, k3, w_post=t["wp2"])
    du, hu = da.swiglu_bwd(da.layer_gemm(b3.dy, t["wd"], b_mn_major=False), u8, with_h=True)
    g = {"wd": da.layer_gemm(hu, b3.dy, a_mn_major=True, out_fp32=True),
         "wu": da.act8_wgrad(k2.xhat8, du, row_scale=t["w2"])}
    b2 = da.block_norm_bwd(b3.dx, da.layer_gemm(du, t["wu"], b_mn_major=False), k2, **kw)
    do = da.layer_gemm(b2.dy, t["wo"], b_mn_major=False)
    g["wo"] = da.layer_gemm(o.view(rows, -1), b2.dy, a_mn_major=True, out_fp32=True)
    dq, dk, dv = da.attn_bwd(q, k, v, o, lse, do.view(o.shape))
    dqkv = torch.cat([dq, dk, dv], dim=2).view(rows, -1)
    g["wqkv"] = da.act8_wgrad(k1.xhat8, dqkv, row_scale=t["w1"])
    b1 = da.block_norm_bwd(b2.dx, da.layer_gemm(dqkv, t["wqkv"], b_mn_major=False), k1, w_pre=t["w1"])
    g.update(x=b1.dx, w1=b1.dw_pre, w2=b2.dw_pre, wp=b2.dw_post, wp2=b3.dw_post, gate=b2.dgate)
    return x2, g


def _decoder_layer_fp64(t, B, T, Hq, Hkv, D, eps=1e-6):
    import oracle
    r, s = 0.9, 0.7
    f1 = ob.norm_fwd(t["x"], w_pre=t["w1"], eps=eps)
    qkv = (f1["h"] @ t["wqkv"]).reshape(B, T, -1, D)
    q, k, v = (np.ascontiguousarray(a) for a in np.split(qkv, [Hq, Hq + Hkv], axis=2))
    o, _ = oracle.attn_fwd(q, k, v, D ** -0.5, True)
    of = o.reshape(B * T, -1)
    y = of @ t["wo"]
    f2 = ob.norm_fwd(t["x"], y, t["gate"], t["wp"], t["w2"], r, s, eps)
    u = f2["h"] @ t["wu"]
    hu = ob.swiglu(u)
    y2 = hu @ t["wd"]
    f3 = ob.norm_fwd(f2["x"], y2, w_post=t["wp2"], eps=eps)

    b3 = ob.norm_bwd(t["dx"], None, None, f3["yhat"], None, f3["rstd_post"], w_post=t["wp2"])
    du = ob.swiglu_grad(b3["dy"] @ t["wd"].T, u)
    b2 = ob.norm_bwd(b3["dx"], du @ t["wu"].T, f2["xhat"], f2["yhat"], f2["rstd_pre"], f2["rstd_post"],
                     t["gate"], t["wp"], t["w2"], r, s)
    do = (b2["dy"] @ t["wo"].T).reshape(o.shape)
    dq, dk, dv, _, _ = oracle.attn_bwd(q, k, v, do, D ** -0.5, True)
    dqkv = np.concatenate([dq, dk, dv], axis=2).reshape(B * T, -1)
    b1 = ob.norm_bwd(b2["dx"], dqkv @ t["wqkv"].T, f1["xhat"], None, f1["rstd_pre"], None,
                     w_pre=t["w1"], block=False)
    return f3["x"], {"wd": hu.T @ b3["dy"], "wu": f2["h"].T @ du, "wo": of.T @ b2["dy"],
                     "wqkv": f1["h"].T @ dqkv, "x": b1["dx"], "w1": b1["dw_pre"], "w2": b2["dw_pre"],
                     "wp": b2["dw_post"], "wp2": b3["dw_post"], "gate": b2["dgate"]}


@pytest.mark.gpu
def test_decoder_layer_from_8_bit_checkpoints_matches_oracle():
    """The operators as a layer uses them, against the same layer in fp64
    without checkpoints.

    A checkpoint of near-normal values has steps of at most 1 / 63.5 of the
    largest of 32, about 2.8 sigma: an rms error of up to 2.8 / 63.5 / sqrt(12)
    = 1.3e-2 of the values.  What a gradient takes from one checkpoint is off by
    that; behind the gated unit two of its inputs are, times slopes up to 1.1
    (2e-2), and the bf16 steps in between (2^-9 rms / sqrt(3) each, and the
    attention's own bar of 1e-2) add 1.1e-2: sqrt(1.3^2 + 2^2 + 1.1^2) = 2.7e-2.
    Held to 3e-2; the stream itself to 1e-2."""
    B, T, Hq, Hkv, D, d, f = 2, 192, 4, 2, 64, 256, 384
    g = _gen(41)
    n = lambda *sh, std=1.0: torch.randn(sh, generator=g) * std
    rows, n3 = B * T, (Hq + 2 * Hkv) * D
    t = {"x": n(rows, d).to(BF), "dx": n(rows, d, std=0.1).to(BF), "wqkv": n(d, n3, std=d ** -0.5).to(BF),
         "wo": n(Hq * D, d, std=(Hq * D) ** -0.5).to(BF), "wu": n(d, 2 * f, std=d ** -0.5).to(BF),
         "wd": n(f, d, std=f ** -0.5).to(BF), "gate": 1 + n(1, d, std=0.2)}
    t.update({w: 1 + n(d, std=0.2) for w in ("w1", "w2", "wp", "wp2")})
    c = {k: v.cuda() for k, v in t.items()}
    x2, got = _decoder_layer(c, B, T, Hq, Hkv, D)
    torch.cuda.synchronize()
    da.check_status()
    ref_x2, ref = _decoder_layer_fp64({k: to_np(v) for k, v in t.items()}, B, T, Hq, Hkv, D)
    assert rel_l2(to_np(x2), ref_x2) <= 1e-2
    for k in ref:
        err = rel_l2(to_np(got[k]).reshape(ref[k].shape), ref[k])
        assert err <= 3e-2, f"{k}: rel-L2 {err:.3g}"
    again, got2 = _decoder_layer(c, B, T, Hq, Hkv, D)
    assert torch.equal(x2, again)
    for k in got:
        assert torch.equal(got[k], got2[k]), k
