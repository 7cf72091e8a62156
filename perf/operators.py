"""The training-block operators as cases to measure: block norms with gate and
residual scale, 8-bit activation checkpoints and the gradients taken from them.

Each case is one call (or, for a checkpoint that is made and read back, the two
calls) of the public entry points, at the shapes of this repository's own
layers (d_model 768 on 4 x 1024 tokens; 1536 on 32 x 1024 tokens; 32 heads of
128 over 8192 positions) and at ragged ones.  ``run`` computes the operators in
elementary torch operations, or with ``own`` through the library.

Formulas, per row of width d, all sums in 32 bits (r = residual scale, s = block
scale, g = gate or its sigmoid, both norms root-mean-square with weight):

    yhat = y * rstd_y,  z = yhat * w_post,  x' = r x + s g z
    xhat = x' * rstd_x,  h = xhat * w_pre
    D  = dx' + rstd_x (dh w_pre - xhat mean(dh w_pre xhat))
    dx = r D,  dz = s g D,  dg = s z D (summed over the rows that share the gate)
    dy = rstd_y (dz w_post - yhat mean(dz w_post yhat))
    dw_pre = sum dh xhat,  dw_post = sum dz yhat

A checkpoint holds int8 values q and, for every 32 consecutive columns of a
row, one byte e: the value is q 2^(e - 127), with e the smallest exponent
(1 at least) for which no |value| exceeds 127 2^(e - 127); rounding to even.
"""
import math

import torch

own = False

GROUP = 32
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The norm before the first block of the smallest batch (1 x 128 tokens): latency.
        _norm("norm_fwd_first_128x768", "norm_fwd", 128, 768, block=False),
        # Between two blocks of the 4 x 1024 layer; what the backward needs kept in 8 bits.
        _norm("norm_fwd_keep8_4096x768", "norm_fwd", 4096, 768, gate="channel", keep8=True),
        # The large layer (32 x 1024 tokens): fp32 residual stream, a gate for every element.
        _norm("norm_fwd_f32_32768x1536", "norm_fwd", 32768, 1536, gate="token", stream="fp32",
              sigmoid=True),
        # One odd-length document at a width that is no power of two; no norm after the block.
        _norm("norm_fwd_ragged_1187x1000", "norm_fwd", 1187, 1000, post=False, gate="channel"),
        # The backward of the 4 x 1024 layer from its 8-bit checkpoints.
        _norm("norm_bwd_from8_4096x768", "norm_bwd", 4096, 768, gate="channel", keep8=True),
        # The backward of the large layer from bf16, one gate row for each of 32 sequences.
        _norm("norm_bwd_seq_32768x1536", "norm_bwd", 32768, 1536, gate="seq32"),
        # The long-context layer's input into 8 bits and back.
        {"name": "act8_round_8192x4096", "op": "act8", "rows": 8192, "d": 4096},
        # Weight gradient of the joined projection from the checkpoint: the 4 x 1024 layer
        # (12 + 2 x 4 heads of 64), the long-context one (32 + 2 x 8 heads of 128), a ragged one.
        {"name": "act8_wgrad_4096x768x1280", "op": "wgrad", "rows": 4096, "d": 768, "n": 1280},
        {"name": "act8_wgrad_8192x4096x6144", "op": "wgrad", "rows": 8192, "d": 4096, "n": 6144},
        {"name": "act8_wgrad_1777x1184x1000", "op": "wgrad", "rows": 1777, "d": 1184, "n": 1000},
        # Gated unit of the 768-wide model with its checkpoint, and the large one's backward from 8 bits.
        {"name": "swiglu_fwd_keep8_4096x2048", "op": "swiglu_fwd", "rows": 4096, "f": 2048,
         "keep8": True},
        {"name": "swiglu_bwd_from8_32768x4096", "op": "swiglu_bwd", "rows": 32768, "f": 4096,
         "keep8": True},
    ]


def _norm(name, op, rows, d, block=True, post=True, pre=True, gate="none", stream="bf16",
          sigmoid=False, keep8=False):
    gate = gate if block else "none"
    return {"name": name, "op": op, "rows": rows, "d": d, "block": block, "post": post and block,
            "pre": pre, "gate": gate, "stream": stream, "sigmoid": sigmoid and gate != "none",
            "keep8": keep8}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_fwd", "norm_bwd", "act8", "wgrad", "swiglu_fwd",
                     "swiglu_bwd"])
    keep8 = rng.random() < 0.5
    if op in ("norm_fwd", "norm_bwd"):
        step = 32 if keep8 else 8
        d = max(step, _log(rng, 32, 8192) // step * step)
        rows = min(_log(rng, 1, 32768), 32768 * 1536 // d)
        gate = rng.choice(["none", "channel", "seq", "token"])
        if gate == "seq":
            n = rng.randint(2, 9)
            rows = max(1, rows // n) * n
            gate = "seq%d" % n
        block = rng.random() < 0.9
        c = _norm("", op, rows, d, block=block, post=rng.random() < 0.7,
                  pre=not block or rng.random() < 0.85, gate=gate, stream=rng.choice(["bf16", "fp32"]),
                  sigmoid=rng.random() < 0.4, keep8=keep8)
        del c["name"]
        return c
    if op == "act8":
        return {"op": op, "rows": _log(rng, 1, 16384), "d": _log(rng, 1, 128) * 32}
    if op == "wgrad":
        return {"op": op, "rows": _log(rng, 1, 8192), "d": _log(rng, 1, 128) * 32,
                "n": _log(rng, 1, 768) * 8}
    return {"op": op, "rows": _log(rng, 1, 32768), "f": _log(rng, 1, 128) * 32, "keep8": keep8}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, rows, d):
    """Unit activations with one wide channel in about fifty (as residual streams have), bf16."""
    x = torch.randn((rows, d), generator=g, device="cuda")
    wide = torch.rand((d,), generator=g, device="cuda") < 0.02
    return (x * torch.where(wide, 12.0, 1.0)).to(torch.bfloat16)


def _weight(g, d):
    return 1.0 + 0.2 * torch.randn((d,), generator=g, device="cuda")


def _quantise(x):
    """(q int8, e uint8) of x in the checkpoint's format."""
    rows, d = x.shape
    v = x.view(rows, d // GROUP, GROUP)
    m, p = torch.frexp(v.abs().amax(dim=-1))  # amax = m 2^p, m in [0.5, 1)
    k = torch.where(m <= 127.0 / 128.0, p - 7, p - 6).clamp(-126, 127)
    q = torch.round(torch.ldexp(v, -k.unsqueeze(-1))).to(torch.int8).view(rows, d)
    return q, (k + 127).to(torch.uint8)


def _values(q, e, dtype=torch.float32):
    """The values that a checkpoint stands for."""
    rows, d = q.shape
    k = e.to(torch.int32).unsqueeze(-1) - 127
    return torch.ldexp(q.view(rows, d // GROUP, GROUP).to(dtype), k).view(rows, d)


def _rstd(x):
    return torch.rsqrt(x.double().square().mean(dim=-1) + EPS).float()


def prepare(case, seed):
    g = _gen(seed)
    op, rows = case["op"], case["rows"]
    s = {"case": case, "op": op}
    if op == "act8":
        s["x"] = _activations(g, rows, case["d"])
    elif op == "wgrad":
        s["q"], s["e"] = _quantise(_activations(g, rows, case["d"]).float())
        s["dy"] = (0.1 * torch.randn((rows, case["n"]), generator=g, device="cuda")).to(torch.bfloat16)
        s["scale"] = _weight(g, case["d"])
    elif op in ("swiglu_fwd", "swiglu_bwd"):
        s["u"] = _activations(g, rows, 2 * case["f"])
        if op == "swiglu_bwd":
            s["dh"] = (0.1 * torch.randn((rows, case["f"]), generator=g, device="cuda")).to(torch.bfloat16)
            if case["keep8"]:
                s["q"], s["e"] = _quantise(s["u"].float())
                del s["u"]
    else:
        _prepare_norm(s, case, g)
    return s


def _prepare_norm(s, case, g):
    rows, d = case["rows"], case["d"]
    stream = torch.float32 if case["stream"] == "fp32" else torch.bfloat16
    s["res_scale"], s["block_scale"] = (0.9, 0.5) if case["block"] else (1.0, 1.0)
    s["w_pre"] = _weight(g, d) if case["pre"] else None
    s["w_post"] = _weight(g, d) if case["post"] else None
    kind = case["gate"]
    s["gate"] = None
    if kind == "token":
        s["gate"] = torch.randn((rows, d), generator=g, device="cuda").to(torch.bfloat16)
    elif kind != "none":
        groups = 1 if kind == "channel" else int(kind[3:])
        s["gate"] = 0.5 * torch.randn((groups, d), generator=g, device="cuda") + 0.5
    x = _activations(g, rows, d)  # the stream: before the block (forward), after it (backward)
    s["x"] = x.to(stream)
    s["y"] = (0.5 * _activations(g, rows, d).float()).to(torch.bfloat16) if case["block"] else None
    if case["op"] == "norm_fwd":
        return
    s["dx_out"] = (0.1 * torch.randn((rows, d), generator=g, device="cuda")).to(stream)
    s["dh"] = ((0.1 * torch.randn((rows, d), generator=g, device="cuda")).to(torch.bfloat16)
               if case["pre"] else None)
    s["rstd_pre"] = _rstd(s["x"]) if case["pre"] else None
    s["rstd_post"] = _rstd(s["y"]) if case["post"] else None
    if case["keep8"]:
        s["xhat8"] = s["yhat8"] = None
        if case["pre"]:
            s["xhat8"] = _quantise(s["x"].float() * s["rstd_pre"].unsqueeze(-1))
        if case["block"]:
            r = s["rstd_post"].unsqueeze(-1) if case["post"] else 1.0
            s["yhat8"] = _quantise(s["y"].float() * r)
        del s["x"], s["y"]


# ------------------------------------------------------------------ plain forms
def _gate_rows(s, rows):
    """The gate of every row in 32 bits (None: none), and its slope by the stored value."""
    g = s["gate"]
    if g is None:
        return None, None
    a = g.float().repeat_interleave(rows // g.shape[0], dim=0)
    if not s["case"]["sigmoid"]:
        return a, torch.ones_like(a)
    a = 1.0 / (1.0 + torch.exp(-a))
    return a, a * (1.0 - a)


def _plain_norm_fwd(s):
    c, out = s["case"], {}
    x = s["x"].float()
    if c["block"]:
        z = s["y"].float()
        if c["post"]:
            out["rstd_post"] = 1.0 / torch.sqrt(z.square().mean(dim=-1) + EPS)
            z = z * out["rstd_post"].unsqueeze(-1)
        if c["keep8"]:
            out["yhat8"] = _values(*_quantise(z)).to(torch.bfloat16)
        if c["post"]:
            z = z * s["w_post"]
        g, _ = _gate_rows(s, c["rows"])
        if g is not None:
            z = g * z
        x = s["res_scale"] * x + s["block_scale"] * z
        out["x"] = x.to(s["x"].dtype)
    if c["pre"]:
        out["rstd_pre"] = 1.0 / torch.sqrt(x.square().mean(dim=-1) + EPS)
        xhat = x * out["rstd_pre"].unsqueeze(-1)
        if c["keep8"]:
            out["xhat8"] = _values(*_quantise(xhat)).to(torch.bfloat16)
        out["h"] = (xhat * s["w_pre"]).to(torch.bfloat16)
    return out


def _hats(s, dtype):
    """xhat and yhat as the backward has them: from the checkpoints, or from the tensors."""
    c, xhat, yhat = s["case"], None, None
    if c["keep8"]:
        xhat = _values(*s["xhat8"], dtype) if c["pre"] else None
        yhat = _values(*s["yhat8"], dtype) if c["block"] else None
        return xhat, yhat
    if c["pre"]:
        xhat = s["x"].to(dtype) * s["rstd_pre"].to(dtype).unsqueeze(-1)
    if c["block"]:
        yhat = s["y"].to(dtype)
        if c["post"]:
            yhat = yhat * s["rstd_post"].to(dtype).unsqueeze(-1)
    return xhat, yhat


def _plain_norm_bwd(s):
    c, out = s["case"], {}
    xhat, yhat = _hats(s, torch.float32)
    d = s["dx_out"].float()
    if c["pre"]:
        dh = s["dh"].float()
        a = dh * s["w_pre"]
        d = d + s["rstd_pre"].unsqueeze(-1) * (a - xhat * (a * xhat).mean(dim=-1, keepdim=True))
        out["dw_pre"] = (dh * xhat).sum(dim=0)
    out["dx"] = ((s["res_scale"] if c["block"] else 1.0) * d).to(s["dx_out"].dtype)
    if c["block"]:
        g, slope = _gate_rows(s, c["rows"])
        dz = s["block_scale"] * d
        if g is not None:
            z = yhat * s["w_post"] if c["post"] else yhat
            dg = dz * z * slope
            groups = s["gate"].shape[0]
            out["dgate"] = dg.view(groups, c["rows"] // groups, c["d"]).sum(dim=1).to(s["gate"].dtype)
            dz = dz * g
        if c["post"]:
            out["dw_post"] = (dz * yhat).sum(dim=0)
            a = dz * s["w_post"]
            dz = s["rstd_post"].unsqueeze(-1) * (a - yhat * (a * yhat).mean(dim=-1, keepdim=True))
        out["dy"] = dz.to(torch.bfloat16)
    return out


def _swiglu_parts(s):
    u = _values(s["q"], s["e"]) if "q" in s else s["u"].float()
    a, b = u.chunk(2, dim=-1)
    return a, b, 1.0 / (1.0 + torch.exp(-a))


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "act8":
        return {"x": _values(*_quantise(s["x"].float())).to(torch.bfloat16)}
    if op == "wgrad":
        return {"dw": s["scale"].unsqueeze(-1) * (_values(s["q"], s["e"]).t() @ s["dy"].float())}
    a, b, sig = _swiglu_parts(s)
    out = {}
    if op == "swiglu_fwd":
        out["h"] = (a * sig * b).to(torch.bfloat16)
        if s["case"]["keep8"]:
            out["u8"] = _values(*_quantise(s["u"].float())).to(torch.bfloat16)
        return out
    dh = s["dh"].float()
    da = dh * b * sig * (1.0 + a * (1.0 - sig))
    out["du"] = torch.cat([da, dh * a * sig], dim=-1).to(torch.bfloat16)
    out["h"] = (a * sig * b).to(torch.bfloat16)  # for the next projection's weight gradient
    return out


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import deterministic_attention_gb300 as da
    c, op, out = s["case"], s["op"], {}
    if op == "norm_fwd":
        x_out, h, kept = da.block_norm_fwd(
            s["x"], s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"],
            res_scale=s["res_scale"], block_scale=s["block_scale"], eps=EPS,
            gate_sigmoid=c["sigmoid"], keep8=c["keep8"])
        if c["block"]:
            out["x"] = x_out
        if c["pre"]:
            out["h"], out["rstd_pre"] = h, kept.rstd_pre
        if c["post"]:
            out["rstd_post"] = kept.rstd_post
        if c["keep8"] and c["pre"]:
            out["xhat8"] = da.act8_unpack(kept.xhat8)
        if c["keep8"] and c["block"]:
            out["yhat8"] = da.act8_unpack(kept.yhat8)
        return out
    if op == "norm_bwd":
        if c["keep8"]:
            kept = da.BlockNormKept(rstd_pre=s["rstd_pre"], rstd_post=s["rstd_post"],
                                    xhat8=s["xhat8"] and da.Act8(*s["xhat8"]),
                                    yhat8=s["yhat8"] and da.Act8(*s["yhat8"]))
        else:
            kept = da.BlockNormKept(rstd_pre=s["rstd_pre"], rstd_post=s["rstd_post"], x=s["x"],
                                    y=s["y"])
        r = da.block_norm_bwd(s["dx_out"], s["dh"], kept, gate=s["gate"], w_post=s["w_post"],
                              w_pre=s["w_pre"], res_scale=s["res_scale"],
                              block_scale=s["block_scale"], gate_sigmoid=c["sigmoid"])
        return {k: v for k, v in r._asdict().items() if v is not None}
    if op == "act8":
        return {"x": da.act8_unpack(da.act8_pack(s["x"]))}
    if op == "wgrad":
        return {"dw": da.act8_wgrad(da.Act8(s["q"], s["e"]), s["dy"], row_scale=s["scale"])}
    if op == "swiglu_fwd":
        if not c["keep8"]:
            return {"h": da.swiglu_fwd(s["u"])}
        h, u8 = da.swiglu_fwd(s["u"], keep8=True)
        return {"h": h, "u8": da.act8_unpack(u8)}
    u = da.Act8(s["q"], s["e"]) if c["keep8"] else s["u"]
    du, h = da.swiglu_bwd(s["dh"], u, with_h=True)
    return {"du": du, "h": h}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    op, rows = case["op"], case["rows"]
    kept = 1.0 + 1.0 / GROUP  # bytes of one checkpointed value
    if op == "act8":
        n = rows * case["d"]
        return {"bytes": 4 * n, "flops": 4 * n}
    if op == "wgrad":
        d, n = case["d"], case["n"]
        return {"bytes": rows * d * kept + 2 * rows * n + 4 * d * n + 4 * d, "flops": 2 * rows * d * n}
    if op == "swiglu_fwd":
        n = rows * case["f"]
        return {"bytes": n * (6 + (2 * kept if case["keep8"] else 0)), "flops": 8 * n}
    if op == "swiglu_bwd":
        n = rows * case["f"]
        return {"bytes": n * ((2 * kept if case["keep8"] else 4) + 2 + 4 + 2), "flops": 16 * n}
    n, d = rows * case["d"], case["d"]
    wide = 4 if case["stream"] == "fp32" else 2
    gates = {"none": 0, "channel": 4 * d, "token": 2 * n}.get(case["gate"])
    gates = 4 * d * int(case["gate"][3:]) if gates is None else gates
    weights = 4 * d * (int(case["pre"]) + int(case["post"]))
    stats = 4 * rows * (int(case["pre"]) + int(case["post"]))
    if op == "norm_fwd":
        b = wide * n + gates + weights + stats + 2 * n * int(case["pre"])
        if case["block"]:
            b += 2 * n + wide * n
        if case["keep8"]:
            b += kept * n * (int(case["pre"]) + int(case["block"]))
        return {"bytes": b, "flops": 12 * n}
    has_x, has_y = case["pre"], case["block"] and (case["post"] or case["gate"] != "none")
    b = 2 * wide * n + 2 * gates + 2 * weights + stats  # dx_out in, dx out, gate and its gradient
    b += 2 * n * int(case["pre"]) + 2 * n * int(case["block"])  # dh in, dy out
    b += ((kept if case["keep8"] else wide) * has_x + (kept if case["keep8"] else 2) * has_y) * n
    return {"bytes": b, "flops": 24 * n}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definition in 64 bits."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "act8":
        return {"x": _exact_round8(s["x"].to(f64))}
    if op == "wgrad":
        x = _exact_values(s["q"], s["e"])
        return {"dw": torch.einsum("td,tn,d->dn", x, s["dy"].to(f64), s["scale"].to(f64))}
    if op in ("swiglu_fwd", "swiglu_bwd"):
        u = _exact_values(s["q"], s["e"]) if "q" in s else s["u"].to(f64)
        if op == "swiglu_fwd":
            a, b = u[:, : case["f"]], u[:, case["f"]:]
            h = torch.sigmoid(a) * a * b
            return {"h": h, "u8": _exact_round8(u)} if case["keep8"] else {"h": h}
        return _exact_by_differentiation(u, s["dh"].to(f64))
    return _exact_norm_fwd(s) if op == "norm_fwd" else _exact_norm_bwd(s)


def _exact_values(q, e):
    return q.double() * torch.exp2(e.double() - 127.0).repeat_interleave(GROUP, dim=1)


def _exact_round8(x):
    """x rounded to the checkpoint's grid: steps of 2^k, k from the group's largest value."""
    big = x.abs().unflatten(1, (-1, GROUP)).amax(dim=-1)
    k = torch.ceil(torch.log2(torch.clamp(big / 127.0, min=2.0 ** -126)))
    k = torch.where(127.0 * torch.exp2(k - 1.0) >= big, k - 1.0, k)  # log2 next to a whole number
    k = torch.where(127.0 * torch.exp2(k) < big, k + 1.0, k).clamp(min=-126.0)
    step = torch.exp2(k).repeat_interleave(GROUP, dim=1)
    return torch.round(x / step) * step


def _exact_by_differentiation(u, dh):
    f = dh.shape[1]
    u = u.detach().requires_grad_(True)
    h = u[:, :f] / (1.0 + torch.exp(-u[:, :f])) * u[:, f:]
    (du,) = torch.autograd.grad(h, u, dh)
    return {"du": du, "h": h.detach()}


def _exact_gate(s):
    g = s["gate"]
    if g is None:
        return None
    g = g.double()
    return torch.sigmoid(g) if s["case"]["sigmoid"] else g


def _exact_norm_fwd(s):
    c, out, x = s["case"], {}, s["x"].double()
    rows, d = x.shape
    if c["block"]:
        y = s["y"].double()
        if c["post"]:
            out["rstd_post"] = (torch.einsum("td,td->t", y, y) / d + EPS) ** -0.5
            y = torch.einsum("td,t->td", y, out["rstd_post"])
        if c["keep8"]:
            out["yhat8"] = _exact_round8(y)
        z = torch.einsum("td,d->td", y, s["w_post"].double()) if c["post"] else y
        g = _exact_gate(s)
        if g is not None:
            z = (z.view(g.shape[0], -1, d) * g.unsqueeze(1)).reshape(rows, d)
        x = out["x"] = torch.add(s["res_scale"] * x, z, alpha=s["block_scale"])
    if c["pre"]:
        out["rstd_pre"] = (torch.einsum("td,td->t", x, x) / d + EPS) ** -0.5
        xhat = torch.einsum("td,t->td", x, out["rstd_pre"])
        if c["keep8"]:
            out["xhat8"] = _exact_round8(xhat)
        out["h"] = torch.einsum("td,d->td", xhat, s["w_pre"].double())
    return out


def _exact_norm_bwd(s):
    c, out, f64 = s["case"], {}, torch.float64
    if c["keep8"]:
        xhat = _exact_values(*s["xhat8"]) if c["pre"] else None
        yhat = _exact_values(*s["yhat8"]) if c["block"] else None
    else:
        xhat, yhat = _hats(s, f64)
    grad = s["dx_out"].to(f64)
    rows, d = grad.shape
    if c["pre"]:
        dh, w = s["dh"].to(f64), s["w_pre"].to(f64)
        along = torch.einsum("td,d,td->t", dh, w, xhat) / d
        grad = grad + (dh * w - along.unsqueeze(1) * xhat) * s["rstd_pre"].to(f64).unsqueeze(1)
        out["dw_pre"] = torch.einsum("td,td->d", dh, xhat)
    out["dx"] = grad * (s["res_scale"] if c["block"] else 1.0)
    if not c["block"]:
        return out
    w = s["w_post"].to(f64) if c["post"] else torch.ones(d, dtype=f64, device=grad.device)
    g = _exact_gate(s)
    grad = grad * s["block_scale"]
    if g is not None:
        n = g.shape[0]
        dg = torch.einsum("gtd,gtd,d->gd", grad.view(n, -1, d), yhat.view(n, -1, d), w)
        out["dgate"] = dg * g * (1.0 - g) if c["sigmoid"] else dg
        grad = (grad.view(n, -1, d) * g.unsqueeze(1)).reshape(rows, d)
    if c["post"]:
        out["dw_post"] = torch.einsum("td,td->d", grad, yhat)
        along = torch.einsum("td,d,td->t", grad, w, yhat) / d
        grad = (grad * w - along.unsqueeze(1) * yhat) * s["rstd_post"].to(f64).unsqueeze(1)
    out["dy"] = grad
    return out
