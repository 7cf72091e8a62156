"""GPU tests of the block norms, 8-bit checkpoints, the weight gradient taken
from one and the gated unit where they can go wrong: kernels that follow one
another closely, gates far from zero, guard bytes around every output.

Tolerances are those of test_gpu_block.py unless a test derives its own.
"""
import numpy as np
import pytest
import torch

import deterministic_attention_gb300 as da
from helpers import to_np
from oracle import block as ob
from test_gpu_block import (BF, EPS, F32, U, _acts, _bwd_refs, _check_bwd, _cuda, _gen, _norm_inputs,
                            _within)

# ------------------------------------------------------------ weight gradient


@pytest.mark.gpu
def test_wgrad_blocks_leave_nothing_behind_for_the_next_kernel():
    """Launches that follow one another closely on two streams, so that blocks
    take over shared memory which a pair has just left: a barrier that such a
    pair's products still reached would be counted wrong.  Few steps (fewer
    than the rings are deep, and a few more), odd pairs' columns included."""
    g = _gen(61)
    q = torch.randn((1, 512, 4, 64), generator=g).to(BF).cuda()
    a = torch.randn((512, 256), generator=g).to(BF).cuda()
    calls = []
    for rows, d, n in ((1, 32, 8), (64, 512, 512), (200, 2432, 1032), (321, 96, 264), (449, 768, 1280)):
        c = da.act8_pack(_acts(g, rows, d).cuda())
        dy = torch.randn((rows, n), generator=g).to(BF).cuda()
        calls.append(lambda c=c, dy=dy: da.act8_wgrad(c, dy))
    calls.append(lambda: da.attn_fwd(q, q, q)[0])
    calls.append(lambda: da.layer_gemm(a, a[:256].contiguous(), out_fp32=True))
    refs = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(40):
        outs = []
        for st in streams:
            with torch.cuda.stream(st):
                outs += [f() for f in calls]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert torch.equal(o, refs[i % len(calls)]), (k, i)
    da.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d,n", [(4096, 768, 1280), (8192, 2432, 512), (512, 96, 264)])
def test_wgrad_is_summed_in_short_runs(rows, d, n):
    """A tensor core's own additions lose up to 3e-7 of a sum of 512 tokens.  The
    runs are added in fp32, so the whole loses no more: at most 3e-7 of each
    run's share, and ceil(rows / 512) roundings of 2^-24, which add up like their
    root (16 runs: 2.4e-7 at worst in the last, 0.6e-7 overall, in quadrature):
    rel-L2 <= sqrt(3^2 + 0.6^2) e-7 < 3.1e-7 whatever the number of rows."""
    x, dy = _acts(_gen(rows), rows, d).cuda(), (0.1 * torch.randn((rows, n), generator=_gen(n))).to(BF).cuda()
    c = da.act8_pack(x)
    ref = da.act8_unpack(c).double().T @ dy.double()
    err = float((da.act8_wgrad(c, dy).double() - ref).norm() / ref.norm())
    assert err <= 3.1e-7, err


# ------------------------------------------------------------ gates far from zero
FAR = [-20.0, -12.0, -8.0, 8.0, 12.0, 20.0]


def _far_gate_inputs(rows, d, G, gdt, stream, post, seed):
    i = _norm_inputs(rows, d, (G, gdt), post, True, stream, seed)
    logits = torch.tensor(FAR)[torch.randint(0, len(FAR), i["gate"].shape, generator=_gen(seed + 1))]
    # A third of the gates as they were; the others at and next to the far logits.
    far = torch.rand(i["gate"].shape, generator=_gen(seed + 2)) < 0.67
    i["gate"] = torch.where(far, logits + 0.1 * i["gate"].float(), i["gate"].float()).to(gdt)
    return i


@pytest.mark.gpu
@pytest.mark.parametrize("gdt", [F32, BF])
@pytest.mark.parametrize("rows,d,G,stream,post", [
    (1, 64, 1, "fp32", True),        # one row: its own gate, nothing summed
    (6, 256, "row", "bf16", True), (7, 2304, "row", "fp32", False),
    (9, 768, 3, "fp32", True), (40, 1536, 1, "bf16", False), (12, 4608, 2, "fp32", True)])
@pytest.mark.parametrize("keep8", [False, True])
def test_sigmoid_gate_keeps_its_slope_when_open_or_shut(rows, d, G, stream, post, gdt, keep8):
    """dgate through sigma' = sigma(x) sigma(-x) at logits up to 20, where sigma
    (1 - sigma) from a rounded sigma has no digits left.  The bound is the one
    for every gate: (rows + 264) u of the magnitudes, which hold sigma' itself.
    (sigma' is within 8 u + |x| u here; 20 and the 64 u of the factors beside
    it are counted with each term, of 264.)"""
    i = _far_gate_inputs(rows, d, G, gdt, stream, post, rows + d)
    c = _cuda(i)
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], res_scale=0.9, block_scale=0.6,
              gate_sigmoid=True)
    _, _, kept = da.block_norm_fwd(c["x"], c["y"], eps=EPS, keep8=keep8, **kw)
    got = da.block_norm_bwd(c["dx_out"], c["dh"], kept, **kw)
    _check_bwd(got, _bwd_refs(i, kept, 0.9, 0.6, True), rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 2])
def test_sigmoid_gate_at_infinite_logits(rows):
    """A gate that is shut or open for good (a mask) has sigma 0 or 1 and a
    slope of zero; a NaN stays in its own columns."""
    d = 64
    gate = torch.zeros((1, d), device="cuda")
    gate[0, :8], gate[0, 8:16], gate[0, 16:24], gate[0, 24] = float("inf"), float("-inf"), -200.0, float("nan")
    gate[0, 32:40] = torch.finfo(F32).min
    x, y = torch.zeros((rows, d), device="cuda"), torch.ones((rows, d), dtype=BF, device="cuda")
    x_out, _, kept = da.block_norm_fwd(x, y, gate=gate, gate_sigmoid=True)
    assert (x_out[:, :8] == 1).all() and (x_out[:, 8:24] == 0).all() and (x_out[:, 32:40] == 0).all()
    assert x_out[:, 24].isnan().all() and (x_out[:, 25:32] == 0.5).all() and (x_out[:, 40:] == 0.5).all()
    g = da.block_norm_bwd(torch.ones_like(x), None, kept, gate=gate, gate_sigmoid=True)
    assert not g.dgate[:, :24].any() and not g.dgate[:, 32:40].any() and g.dgate[:, 24].isnan().all()
    assert (g.dgate[:, 25:32] == 0.25 * rows).all() and (g.dy[:, :8] == 1).all() and not g.dy[:, 8:24].any()


@pytest.mark.gpu
@pytest.mark.parametrize("gdt", [F32, BF])
def test_sigmoid_of_shut_gates_is_as_good_as_of_open_ones(gdt):
    """sigma itself, read from an fp32 stream (r = 0, y = 1: x' = s sigma), over
    -87 .. 87.  Its relative error: the power of two 4 u (2^-22), its exponent's
    rounding carried along (1 u), the sum 1 u, the quotient 4 u (two units in
    the last place), the last product 1 u: 11 u, held to 16 u at any logit."""
    rows, d = 40, 1024
    gate = ((torch.rand((rows, d), generator=_gen(71)) - 0.5) * 174.0).to(gdt)
    x, y = torch.zeros((rows, d)), torch.ones((rows, d), dtype=BF)
    x_out, _, kept = da.block_norm_fwd(x.cuda(), y.cuda(), gate=gate.cuda(), res_scale=0.0,
                                       gate_sigmoid=True)
    ref = ob.sigmoid(to_np(gate))
    _within("sigma", to_np(x_out), ref, ref, 16, 0.0)
    # Its slope: two more factors sigma, three roundings: 16 u + 11 u + 3 u.
    g = da.block_norm_bwd(torch.ones((rows, d), device="cuda"), None, kept, gate=gate.cuda(),
                          gate_sigmoid=True)
    ref = ref * ob.sigmoid(-to_np(gate))
    _within("slope", to_np(g.dgate), ref, ref, 30, 2.0 ** -8 if gdt == BF else 0.0)


# ------------------------------------------------------------ gated unit
@pytest.mark.gpu
@pytest.mark.parametrize("from8", [False, True])
def test_swiglu_far_below_zero(from8):
    """sigma(a) below 2^-126, where it is no normal fp32 number, times a b large
    enough to bring the product back among bf16's: h and du keep the relative
    accuracy of every other argument.  (2^-8 for the store; exp's rounded
    argument |a| 2^-24, twice for the root squared, and a few units beside it:
    400 u of the magnitudes, far below the store's; 1.2e-38: bf16's smallest
    normal number, below which a store has fewer bits.)"""
    a = torch.tensor([-80.0, -87.0, -87.5, -88.0, -88.5, -90.0, -95.0, -100.0, -120.0, -150.0, -170.0, -3e38]
                     + [20.0, 88.0, 90.0, 120.0]).to(BF)
    b = torch.tensor([1e30, 1e38, 3e38, -2e36]).to(BF)
    f = 32 * len(b)
    u = torch.zeros((len(a), 2 * f))
    for j, v in enumerate(b):
        # (32 equal values: a group of a checkpoint each)
        u[:, 32 * j:32 * j + 32] = a.float()[:, None]
        u[:, f + 32 * j:f + 32 * j + 32] = v.float() * torch.where(a.float() > 0, 1e-30, 1.0)[:, None]
    u = u.to(BF)
    dh = torch.full((len(a), f), -0.75, dtype=BF)
    dh[:, ::2] = 1.5
    c = da.act8_pack(u.cuda()) if from8 else u.cuda()
    u64 = ob.act8_values(c.q.cpu().numpy(), c.e.cpu().numpy()) if from8 else to_np(u)
    du, h = da.swiglu_bwd(dh.cuda(), c, with_h=True)
    ref, dref = ob.swiglu(u64), ob.swiglu_grad(to_np(dh), u64)
    x, y = np.split(u64, 2, axis=-1)
    s, g = ob.sigmoid(x), np.abs(to_np(dh))
    mag = np.concatenate([g * np.abs(y) * s * (1 + np.abs(x) * ob.sigmoid(-x)), g * np.abs(x) * s], -1)
    for name, got, want, m in (("h", h, ref, np.abs(ref)), ("du", du, dref, mag)):
        bound = 2.0 ** -8 * np.abs(want) + 400 * U * m + 1.2e-38
        err = np.abs(to_np(got) - want)
        assert np.isfinite(to_np(got)).all() and (err <= bound).all(), (name, float((err / bound).max()))
    if not from8:
        assert torch.equal(da.swiglu_fwd(u.cuda()), h)


# ------------------------------------------------------------ gate rows shared by few rows
@pytest.mark.gpu
@pytest.mark.parametrize("rows,G,d,stream", [(1000, 100, 768, "bf16"), (630, 90, 64, "fp32"),
                                             (1824, 304, 2304, "bf16"), (1830, 305, 768, "bf16")])
@pytest.mark.parametrize("keep8", [False, True])
def test_gate_rows_shared_by_few_rows(rows, G, d, stream, keep8):
    """Slices of one to three rows, uneven ones, and whole gate rows per item."""
    i = _norm_inputs(rows, d, (G, F32), True, True, stream, rows + G)
    c = _cuda(i)
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], res_scale=0.9, block_scale=0.6)
    _, _, kept = da.block_norm_fwd(c["x"], c["y"], eps=EPS, keep8=keep8, **kw)
    got = da.block_norm_bwd(c["dx_out"], c["dh"], kept, **kw)
    _check_bwd(got, _bwd_refs(i, kept, 0.9, 0.6, False), rows)
    again = da.block_norm_bwd(c["dx_out"], c["dh"], kept, **kw)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


# ------------------------------------------------------------ waits that run out
@pytest.mark.gpu
def test_waits_that_run_out_are_reported_by_name_and_cleared():
    """The bounded waits of the weight gradient and of the norm backward, on a
    barrier nothing completes: each sets its own status word, the host reads
    which, and the same context then computes as before."""
    i = _cuda(_norm_inputs(100, 768, (1, F32), True, True, "bf16", 73))
    kw = dict(gate=i["gate"], w_post=i["w_post"], w_pre=i["w_pre"])
    _, h, kept = da.block_norm_fwd(i["x"], i["y"], keep8=True, **kw)

    def both():
        return [*da.block_norm_bwd(i["dx_out"], i["dh"], kept, **kw), da.act8_wgrad(kept.xhat8, h)]
    ref = both()
    da.check_status()
    da.selftest_wait_timeout(2_000_000)
    with pytest.raises(da.DetAttnError, match="act8_wgrad 1, block_norm_bwd 1") as e:
        da.check_status()
    assert e.value.code == -7
    da.check_status()
    for a, b in zip(ref, both()):
        assert torch.equal(a, b)
    da.check_status()


# ------------------------------------------------------------ guard bytes
class _Guards:
    """Outputs with 256 guard bytes before and after; `shift` bytes off alignment."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype, shift=0):
        size = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.bufs.append((raw, 256 + shift, size))
        return raw[256 + shift:256 + shift + size]

    def check(self):
        for raw, at, size in self.bufs:
            assert (raw[:at] == 0xA5).all() and (raw[at + size:] == 0xA5).all(), size


def _same(got, ref):
    """Raw bytes of a guarded output against the binding's tensor."""
    assert torch.equal(got, ref.contiguous().view(-1).view(torch.uint8).view(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [(1, F32), ("row", BF), (67, F32)])
@pytest.mark.parametrize("rows,d,stream", [(67, 1056, "bf16"), (134, 96, "fp32"), (67, 4608, "bf16")])
@pytest.mark.parametrize("keep8", [False, True])
def test_norms_write_every_output_and_nothing_beside_it(rows, d, stream, gate, keep8):
    """All outputs of both norms through the C entry points, workspace included:
    the same bytes as through the binding, guard bytes untouched, the exponent
    bytes at odd addresses and the statistics four bytes off."""
    G = rows if gate[0] == "row" else gate[0]
    i = _cuda(_norm_inputs(rows, d, gate, True, True, stream, rows + d))
    kw = dict(gate=i["gate"], w_post=i["w_post"], w_pre=i["w_pre"])
    x_out, h, kept = da.block_norm_fwd(i["x"], i["y"], keep8=keep8, **kw)
    ref = da.block_norm_bwd(i["dx_out"], i["dh"], kept, **kw)
    g, p = _Guards(), (lambda t: None if t is None else t.data_ptr())
    st, f32 = i["x"].dtype, stream == "fp32"
    out = {"x": g((rows, d), st), "h": g((rows, d), BF), "ro": g((rows,), F32, 4), "rp": g((rows,), F32, 4)}
    for n in ("y", "x"):
        out[n + "q"] = g((rows, d), torch.int8) if keep8 else None
        out[n + "e"] = g((rows, d // 32), torch.uint8, 3) if keep8 else None
    L, flags = da.lib(), (int(f32), int(gate[1] == F32), 0)
    rc = L.block_norm_fwd(p(i["x"]), p(i["y"]), p(i["gate"]), p(i["w_post"]), p(i["w_pre"]), p(out["x"]),
                          p(out["h"]), p(out["ro"]), p(out["rp"]), p(out["yq"]), p(out["ye"]), p(out["xq"]),
                          p(out["xe"]), rows, d, G, *flags, 1.0, 1.0, EPS, None)
    assert rc == 0, da.last_error()
    torch.cuda.synchronize()
    for a, b in ((out["x"], x_out), (out["h"], h), (out["ro"], kept.rstd_post), (out["rp"], kept.rstd_pre)):
        _same(a, b)
    if keep8:
        for n, c in (("y", kept.yhat8), ("x", kept.xhat8)):
            _same(out[n + "q"], c.q)
            _same(out[n + "e"], c.e)
    need = da.block_norm_bwd_workspace_bytes(rows, d, G)
    ws = g((need,), torch.uint8)
    grads = [g((rows, d), st), g((rows, d), BF), g((G, d), gate[1]), g((d,), F32), g((d,), F32)]
    rc = L.block_norm_bwd(p(i["dx_out"]), p(i["dh"]), None if keep8 else p(x_out),
                          None if keep8 else p(i["y"]), p(out["xq"]), p(out["xe"]), p(out["yq"]),
                          p(out["ye"]), p(i["gate"]), p(i["w_post"]), p(i["w_pre"]), p(out["ro"]),
                          p(out["rp"]), *(p(t) for t in grads), p(ws), need, rows, d, G, *flags, 1.0, 1.0,
                          None)
    assert rc == 0, da.last_error()
    torch.cuda.synchronize()
    for a, b in zip(grads, ref):
        _same(a, b)
    g.check()
    da.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d,n", [(1777, 1184, 504), (300, 96, 264), (129, 2496, 2056)])
def test_wgrad_writes_every_output_and_nothing_beside_it(rows, d, n):
    """Cut tiles (the partial tiles and their sum under guards), whole ones, and
    more whole ones than pairs of blocks, ragged both ways; the exponent bytes
    at odd addresses."""
    need = da.act8_wgrad_workspace_bytes(rows, d, n)
    assert (need > 0) == (rows > 1000)
    g = _Guards()
    x, dy = _acts(_gen(79), rows, d).cuda(), torch.randn((rows, n), generator=_gen(80)).to(BF).cuda()
    ref = da.act8_wgrad(da.act8_pack(x), dy)
    q, e = g((rows, d), torch.int8), g((rows, d // 32), torch.uint8, 1)
    L = da.lib()
    assert L.act8_pack(x.data_ptr(), q.data_ptr(), e.data_ptr(), rows, d, None) == 0
    back = g((rows, d), BF)
    assert L.act8_unpack(q.data_ptr(), e.data_ptr(), back.data_ptr(), rows, d, None) == 0
    dw, ws = g((d, n), F32), g((max(need, 16),), torch.uint8)
    assert L.act8_wgrad(q.data_ptr(), e.data_ptr(), dy.data_ptr(), None, dw.data_ptr(), ws.data_ptr(), need,
                        rows, d, n, None) == 0, da.last_error()
    torch.cuda.synchronize()
    _same(dw, ref)
    _same(back, da.act8_unpack(da.act8_pack(x)))
    g.check()
    da.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,f", [(1, 32), (67, 1056), (130, 96)])
def test_swiglu_writes_every_output_and_nothing_beside_it(rows, f):
    g, L = _Guards(), da.lib()
    u, dh = _acts(_gen(81), rows, 2 * f).cuda(), torch.randn((rows, f), generator=_gen(82)).to(BF).cuda()
    href, c = da.swiglu_fwd(u, keep8=True)
    h, q, e = g((rows, f), BF), g((rows, 2 * f), torch.int8), g((rows, f // 16), torch.uint8, 5)
    assert L.swiglu_fwd(u.data_ptr(), h.data_ptr(), q.data_ptr(), e.data_ptr(), rows, f, None) == 0
    for from8 in (False, True):
        duref, href2 = da.swiglu_bwd(dh, c if from8 else u, with_h=True)
        du, h2 = g((rows, 2 * f), BF), g((rows, f), BF)
        kept = (None, q.data_ptr(), e.data_ptr()) if from8 else (u.data_ptr(), None, None)
        assert L.swiglu_bwd(dh.data_ptr(), *kept, du.data_ptr(), h2.data_ptr(), rows, f, None) == 0
        torch.cuda.synchronize()
        _same(du, duref)
        _same(h2, href2)
    for a, b in ((h, href), (q, c.q), (e, c.e)):
        _same(a, b)
    g.check()


# ------------------------------------------------------------ forms of the norms' calls
@pytest.mark.gpu
@pytest.mark.parametrize("rows,d,gate,sig,post,stream", [
    (37, 768, (1, F32), False, True, "bf16"), (37, 768, ("row", BF), True, True, "fp32"),
    (40, 1536, (4, F32), True, False, "fp32"), (21, 2304, None, False, True, "bf16"),
    (50, 8, (1, F32), False, True, "bf16"), (9, 8192, None, False, False, "fp32")])
@pytest.mark.parametrize("keep8", [False, True])
def test_nothing_comes_back_along_the_stream(rows, d, gate, sig, post, stream, keep8):
    """dx_out = None behind a block (the last norm of a model): the gradients
    with a dx_out of zeros.  From checkpoints the stream is then taken as bf16."""
    if keep8 and d % 32:
        pytest.skip("a checkpoint needs a multiple of 32 columns")
    i = _norm_inputs(rows, d, gate, post, True, stream, 3 * rows + d)
    c = _cuda(i)
    kw = dict(gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], res_scale=0.9, block_scale=0.6,
              gate_sigmoid=sig)
    _, _, kept = da.block_norm_fwd(c["x"], c["y"], eps=EPS, keep8=keep8, **kw)
    got = da.block_norm_bwd(None, c["dh"], kept, **kw)
    assert got.dx.dtype == (BF if keep8 else i["x"].dtype)
    i["dx_out"] = None
    _check_bwd(got, _bwd_refs(i, kept, 0.9, 0.6, sig), rows)


@pytest.mark.gpu
@pytest.mark.parametrize("keep8", [False, True])
def test_has_block_says_what_kept_does_not(keep8):
    """A block without gate or norm after it needs no y: with has_block its
    gradient comes without y being kept; without, there is no dy and the
    scales are not used."""
    i = _norm_inputs(70, 1056, None, False, True, "bf16", 83)
    c = _cuda(i)
    _, _, kept = da.block_norm_fwd(c["x"], c["y"], w_pre=c["w_pre"], keep8=keep8)
    kw = dict(w_pre=c["w_pre"], res_scale=0.9, block_scale=0.6)
    ref = da.block_norm_bwd(c["dx_out"], c["dh"], kept, **kw)
    less = kept._replace(y=None, yhat8=None)
    for a, b in zip(da.block_norm_bwd(c["dx_out"], c["dh"], less, has_block=True, **kw), ref):
        assert (a is None and b is None) or torch.equal(a, b)
    alone = da.block_norm_bwd(c["dx_out"], c["dh"], kept, has_block=False, **kw)
    plain = da.block_norm_bwd(c["dx_out"], c["dh"], less, w_pre=c["w_pre"])
    assert alone.dy is None and torch.equal(alone.dx, plain.dx) and torch.equal(alone.dw_pre, plain.dw_pre)
    with pytest.raises(ValueError, match="belong to"):
        da.block_norm_bwd(c["dx_out"], c["dh"], kept, has_block=False, w_post=c["w_pre"], **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [None, (1, F32), ("row", BF)])
def test_gradients_may_overwrite_what_they_come_from(gate):
    """dx over dx_out and dy over y, through the C entry point."""
    rows, d = 1300, 1536
    i = _cuda(_norm_inputs(rows, d, gate, True, True, "bf16", 89))
    kw = dict(gate=i["gate"], w_post=i["w_post"], w_pre=i["w_pre"])
    x_out, _, kept = da.block_norm_fwd(i["x"], i["y"], **kw)
    ref = da.block_norm_bwd(i["dx_out"], i["dh"], kept, **kw)
    p = lambda t: None if t is None else t.data_ptr()
    G = 1 if gate is None else i["gate"].shape[0]
    dgate, dwo, dwp = (None if t is None else torch.empty_like(t)
                       for t in (i["gate"], i["w_post"], i["w_pre"]))
    ws = torch.empty(da.block_norm_bwd_workspace_bytes(rows, d, G), dtype=torch.uint8, device="cuda")
    rc = da.lib().block_norm_bwd(p(i["dx_out"]), p(i["dh"]), p(x_out), p(i["y"]), None, None, None, None,
                                 p(i["gate"]), p(i["w_post"]), p(i["w_pre"]), p(kept.rstd_post),
                                 p(kept.rstd_pre), p(i["dx_out"]), p(i["y"]), p(dgate), p(dwo), p(dwp),
                                 p(ws), ws.numel(), rows, d, G, 0, int(gate == (1, F32)), 0, 1.0, 1.0, None)
    assert rc == 0, da.last_error()
    torch.cuda.synchronize()
    for a, b in zip((i["dx_out"], i["y"], dgate, dwo, dwp), ref):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.gpu
def test_a_gate_row_is_shared_by_consecutive_rows():
    """[B, d] and [B, 1, d] gates are one row per sequence of a [B, T, d] stream;
    [B, T, d] one per token."""
    B, T, d = 3, 5, 64
    g = _gen(97)
    x, y = torch.zeros((B, T, d), device="cuda"), torch.ones((B, T, d), dtype=BF, device="cuda")
    for shape in ((B, d), (B, 1, d), (B, T, d), (d,), (1, 1, d)):
        gate = torch.randn(shape, generator=g).cuda()
        want = (gate[:, None] if shape == (B, d) else gate).expand(B, T, d)
        assert torch.equal(da.block_norm_fwd(x, y, gate=gate)[0], want)


@pytest.mark.gpu
def test_two_host_threads_at_once():
    """First calls of kernels not used before, from two threads on two streams."""
    import threading
    outs, errs = {}, []
    i = _cuda(_norm_inputs(60, 5120, (1, F32), True, True, "fp32", 101))
    dy = torch.randn((60, 40), generator=_gen(103)).to(BF).cuda()
    torch.cuda.synchronize()

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    kw = dict(gate=i["gate"], w_post=i["w_post"], w_pre=i["w_pre"])
                    _, h, kept = da.block_norm_fwd(i["x"], i["y"], keep8=True, **kw)
                    got = da.block_norm_bwd(i["dx_out"], i["dh"], kept, **kw)
                    dw = da.act8_wgrad(kept.xhat8, dy)
                    with pytest.raises(da.DetAttnError, match="eps"):
                        da.block_norm_fwd(i["x"], w_pre=i["w_pre"], eps=-1.0)
                torch.cuda.current_stream().synchronize()
                outs[k] = [h, *got, dw]
        except BaseException as e:  # noqa: BLE001
            errs.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errs, errs
    for a, b in zip(outs[0], outs[1]):
        assert torch.equal(a, b)
    da.check_status()
