"""The ends of a training step as cases to measure: rotary positions before the
attention, the output projection's softmax cross entropy, the orthogonalised
update of a weight matrix.

Each case is one call of the public entry points, at the shapes of this
repository's own layers (12 + 4 heads of 64 over 4 x 1024 tokens; 24 + 24 heads
of 64; 32 + 8 heads of 128 over long sequences; d_model 768 and 1536; 50,257 words,
padded to 50,432) and at ragged ones.  ``run`` computes the operators in
elementary torch operations, or with ``own`` through the library.

Rotary positions: with theta_i the angle per position of pair i, t a token's
position, m a factor of the scaling, for every head

    (a, b) -> m (a cos t theta_i - b sin t theta_i,  b cos t theta_i + a sin t theta_i)

where (a, b) are components (2 i, 2 i + 1) (interleaved) or (i, i + rot / 2)
(halves) of the first rot components; the others pass.  The backward turns by
the opposite angle.

Cross entropy of x [N, d] with the output weight w [V, d]: z = x w^T,
lse_n = ln sum_v exp z_nv, loss_n = lse_n - z_n,target (0 for a row without a
target, target < 0).  Backward, g the gradient of loss (0 without a target), e
that of lse: dz_nv = (g_n + e_n) exp(z_nv - lse_n) - g_n [v = target_n],
dx = dz w, dw = dz^T x.

Orthogonalised update of a gradient g [m, n]: momentum M <- beta M + g, u = g +
beta M (u = g without momentum), X = u / (|u| + eps), |u| the Frobenius norm, then five times

    X <- a X + b (X X^T) X + c (X X^T)^2 X      (by columns where m > n)
"""
import math

import torch

own = False

BASE = 10000.0
BETA, EPS = 0.95, 1e-7
NS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One new token for each of 8 sequences, far into a scaled context: latency.
        _rope("rope_step_8x1_40h128", 8, 1, 32, 8, 128, scaling="ramp", far=131072, joined=True),
        # Q and K of the 4 x 1024 layer, where its joined projection left them.
        _rope("rope_fwd_4x1024_16h64", 4, 1024, 12, 4, 64, joined=True),
        # Gradients of the wide layer (24 + 24 heads), half of each head turned, in fp32; odd length.
        _rope("rope_bwd_part_5x777_48h64", 5, 777, 24, 24, 64, rot=32, interleaved=True, dtype="fp32",
              backward=True),
        # One long document, the long-context layer's heads, bands of wavelengths scaled.
        _rope("rope_fwd_1x65536_40h128", 1, 65536, 32, 8, 128, scaling="bands"),
        # Loss of the smallest batch (1 x 128 tokens) over the whole vocabulary.
        _ce("ce_fwd_128x768x50257", "ce_fwd", 128, 768, 50257),
        # Loss of the large model's step: 32 x 1024 tokens.
        _ce("ce_fwd_32768x1536x50432", "ce_fwd", 32768, 1536, 50432, no_target=0.1),
        # Gradients of one odd-length document.
        _ce("ce_bwd_1187x768x50257", "ce_bwd", 1187, 768, 50257),
        # Gradients of the 4 x 1024 step; a tenth of the tokens have no target.
        _ce("ce_bwd_4096x768x50432", "ce_bwd", 4096, 768, 50432, no_target=0.1),
        # Gradients of the large step, with one for lse (a penalty on its size).
        _ce("ce_bwd_32768x1536x50432", "ce_bwd", 32768, 1536, 50432, dlse=True),
        # One weight of the 768-wide layer: latency of the products one after another.
        _muon("muon_1x768x768", 1, 768, 768, dtype="fp32"),
        # The joined projections (12 + 2 x 4 heads of 64) of twelve layers in one call.
        _muon("muon_12x768x1280", 12, 768, 1280),
        # The joined projection of the long-context layer (32 + 2 x 8 heads of 128).
        _muon("muon_1x4096x6144", 1, 4096, 6144),
    ]


def _rope(name, B, T, hq, hkv, D, rot=0, interleaved=False, dtype="bf16", backward=False,
          scaling="none", far=0, joined=False):
    return {"name": name, "op": "rope", "B": B, "T": T, "hq": hq, "hkv": hkv, "D": D, "rot": rot or D,
            "interleaved": interleaved, "dtype": dtype, "backward": backward, "scaling": scaling,
            "far": far, "joined": joined}


def _ce(name, op, N, d, V, no_target=0.0, dlse=False):
    return {"name": name, "op": op, "N": N, "d": d, "V": V, "no_target": no_target, "dlse": dlse}


def _muon(name, batch, m, n, dtype="bf16", momentum=True):
    return {"name": name, "op": "muon", "batch": batch, "m": m, "n": n, "dtype": dtype,
            "momentum": momentum}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "ce_fwd", "ce_bwd", "muon", "muon"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128])
        hkv = rng.choice([1, 2, 4, 8, 12])
        hq = hkv * rng.choice([1, 2, 3, 4])
        B = _log(rng, 1, 16)
        T = _log(rng, 1, max(1, 65536 * 40 * 128 // (B * (hq + hkv) * D)))
        T = min(T, 65536)
        scaling = rng.choice(["none", "linear", "ramp", "bands"])
        c = _rope("", B, T, hq, hkv, D, rot=rng.choice([D, D, D // 2, D // 4]),
                  interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                  backward=rng.random() < 0.5, scaling=scaling,
                  far=0 if rng.random() < 0.5 else _log(rng, 4096, 1048576), joined=rng.random() < 0.5)
    elif op == "muon":
        batch = _log(rng, 1, 16)
        n = _log(rng, 16, 512) * 8
        m = min(_log(rng, 128, 4096), 4096 * 6144 // (batch * n))
        c = _muon("", batch, max(128, m), n, dtype=rng.choice(["bf16", "fp32"]),
                  momentum=rng.random() < 0.7)
    else:
        d = _log(rng, 32, 192) * 8
        c = _ce("", op, _log(rng, 1, 16384), d, _log(rng, 1000, 50432),
                no_target=rng.choice([0.0, 0.1, 0.5]), dlse=op == "ce_bwd" and rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return std * torch.randn(shape, generator=g, device="cuda")


def _freqs(rot, scaling, factor=16.0, context=8192):
    """(angles per position in 64 bits [rot / 2], factor m) as a model's configuration gives them."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = BASE ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    turns = context * f / (2.0 * math.pi)  # turns within the context that the model was trained on
    if scaling == "bands":  # below one turn divided, above four kept, between in proportion
        keep = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor), 1.0
    if scaling == "ramp":  # the same between one and 32 turns, in proportion to the pair's number
        at = lambda r: rot * math.log(context / (r * 2.0 * math.pi)) / (2.0 * math.log(BASE))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "rope":
        _prepare_rope(s, case, g)
    elif case["op"] == "muon":
        _prepare_muon(s, case, g)
    else:
        _prepare_ce(s, case, g)
    return s


def _prepare_rope(s, case, g):
    B, T, hq, hkv, D = (case[k] for k in ("B", "T", "hq", "hkv", "D"))
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    if case["joined"]:  # views into the joined projection [B, T, Q heads | K heads | V heads]
        qkv = torch.empty((B, T, hq + 2 * hkv, D), dtype=dtype, device="cuda").normal_(generator=g)
        s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv]
    else:
        s["q"] = torch.empty((B, T, hq, D), dtype=dtype, device="cuda").normal_(generator=g)
        s["k"] = torch.empty((B, T, hkv, D), dtype=dtype, device="cuda").normal_(generator=g)
    s["freqs"], s["mscale"] = _freqs(case["rot"], case["scaling"])
    s["positions"] = None  # t = 0 .. T - 1 in every sequence
    if case["far"]:
        start = torch.randint(0, case["far"], (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = (start + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()


def _prepare_ce(s, case, g):
    N, d, V = case["N"], case["d"], case["V"]
    # A normed stream against weights of the usual spread; the target's word is more
    # likely than the others, as in training.
    w = _randn(g, V, d, std=0.02)
    words = (V * torch.rand((N,), generator=g, device="cuda").pow(3)).to(torch.int64).clamp(max=V - 1)
    x = _randn(g, N, d) + 3.0 * w[words] / 0.02 / math.sqrt(d)
    s["x"], s["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
    none = torch.rand((N,), generator=g, device="cuda") < case["no_target"]
    s["targets"] = torch.where(none, -100, words).to(torch.int32)
    if case["op"] == "ce_fwd":
        return
    z = _logits(s)
    s["lse"] = torch.logsumexp(z, dim=1)
    del z
    s["dloss"] = torch.full((N,), 1.0 / max(1, int((~none).sum())), device="cuda")
    s["dlse"] = 1e-4 * s["lse"] / N if case["dlse"] else None


def _prepare_muon(s, case, g):
    shape = (case["batch"], case["m"], case["n"])
    # A gradient: a few directions that many tokens share, and what is each token's own.
    def grad():
        r = 8
        shared = _randn(g, case["batch"], case["m"], r) @ _randn(g, case["batch"], r, case["n"])
        return 1e-4 * (_randn(g, *shape) + 0.5 * shared / math.sqrt(r))

    s["g"] = grad().to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
    s["momentum"] = 5.0 * grad() if case["momentum"] else None


# ------------------------------------------------------------------ plain forms
def _plain_rope(x, s):
    c = s["case"]
    B, T, _, D = x.shape
    rot = c["rot"]
    t = s["positions"]
    if t is None:
        t = torch.arange(T, device=x.device).expand(B, T)
    angle = t.double().unsqueeze(-1) * s["freqs"] * (-1.0 if c["backward"] else 1.0)
    cos = (torch.cos(angle) * s["mscale"]).float().unsqueeze(2)
    sin = (torch.sin(angle) * s["mscale"]).float().unsqueeze(2)
    f = x.float()
    a, b = (f[..., 0:rot:2], f[..., 1:rot:2]) if c["interleaved"] else (f[..., :rot // 2], f[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), dim=-1).flatten(-2) if c["interleaved"] else torch.cat((u, v), dim=-1)
    return torch.cat((turned.to(x.dtype), x[..., rot:]), dim=-1)


def _logits(s):
    return s["x"].float() @ s["w"].float().t()


def _plain_ce_fwd(s):
    z = _logits(s)
    top = z.amax(dim=1)
    z -= top.unsqueeze(1)
    t = s["targets"].to(torch.int64)
    zt = z.gather(1, t.clamp(min=0).unsqueeze(1)).squeeze(1)
    ln = torch.log(z.exp_().sum(dim=1))
    return {"loss": torch.where(t >= 0, ln - zt, 0.0), "lse": top + ln}


def _plain_ce_bwd(s):
    t = s["targets"].to(torch.int64)
    g = torch.where(t >= 0, s["dloss"], 0.0)
    z = _logits(s)
    z -= s["lse"].unsqueeze(1)
    z.exp_()
    z *= (g if s["dlse"] is None else g + s["dlse"]).unsqueeze(1)
    z.scatter_add_(1, t.clamp(min=0).unsqueeze(1), -g.unsqueeze(1))
    dx = (z @ s["w"].float()).to(torch.bfloat16)
    return {"dx": dx, "dw": (z.t() @ s["x"].float()).to(torch.bfloat16)}


def _plain_muon(s):
    g = s["g"].float()
    out = {}
    if s["momentum"] is not None:
        s["momentum"].mul_(BETA).add_(g)
        g = g + BETA * s["momentum"]
        out["momentum"] = s["momentum"]
    x = g / (g.double().square().sum(dim=(1, 2), keepdim=True).sqrt().float() + EPS)
    wide = x.shape[1] <= x.shape[2]
    x = _orthogonal(x if wide else x.mT)
    out["o"] = (x if wide else x.mT.contiguous()).to(torch.bfloat16)
    return out


def _orthogonal(x):
    a, b, c = NS
    for _ in range(NS_STEPS):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x


def run(state):
    c, s = state["case"], state
    if own:
        return _own(s)
    if c["op"] == "rope":
        return {"q": _plain_rope(s["q"], s), "k": _plain_rope(s["k"], s)}
    if c["op"] == "ce_fwd":
        return _plain_ce_fwd(s)
    if c["op"] == "ce_bwd":
        return _plain_ce_bwd(s)
    return _plain_muon(s)


# ------------------------------------------------------------------ through the library
def _own(s):
    import deterministic_attention_gb300 as da
    c = s["case"]
    if c["op"] == "rope":
        call = da.rope_bwd if c["backward"] else da.rope_fwd
        q, k = call(s["q"], s["k"], s["freqs"], positions=s["positions"], interleaved=c["interleaved"],
                    mscale=s["mscale"])
        return {"q": q, "k": k}
    if c["op"] == "ce_fwd":
        loss, lse = da.linear_ce_fwd(s["x"], s["w"], s["targets"])
        return {"loss": loss, "lse": lse}
    if c["op"] == "ce_bwd":
        dx, dw = da.linear_ce_bwd(s["x"], s["w"], s["targets"], s["lse"], s["dloss"], dlse=s["dlse"])
        return {"dx": dx, "dw": dw}
    o = da.muon_update(s["g"], momentum=s["momentum"], beta=BETA, steps=NS_STEPS, eps=EPS)
    return {"o": o} if s["momentum"] is None else {"o": o, "momentum": s["momentum"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["B"] * case["T"] * (case["hq"] + case["hkv"]) * case["D"]
        wide = 4 if case["dtype"] == "fp32" else 2
        b = 2 * wide * n + 4 * case["rot"] + (4 * case["B"] * case["T"] if case["far"] else 0)
        return {"bytes": b, "flops": 3 * n * case["rot"] // case["D"]}
    if op == "muon":
        batch, lo, hi = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
        n = batch * lo * hi
        b = (4 if case["dtype"] == "fp32" else 2) * n + (8 * n if case["momentum"] else 0) + 2 * n
        # Half of each symmetric product, the whole of the last.
        return {"bytes": b, "flops": NS_STEPS * batch * (lo * lo * hi + lo ** 3 + 2 * lo * lo * hi)}
    N, d, V = case["N"], case["d"], case["V"]
    if op == "ce_fwd":
        return {"bytes": 2 * (N + V) * d + 12 * N, "flops": 2 * N * d * V}
    return {"bytes": 4 * (N + V) * d + 12 * N + (4 * N if case["dlse"] else 0), "flops": 6 * N * d * V}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definition in 64 bits."""
    op = case["op"]
    # Products in 64 bits run at about a TFLOP/s; what would take over 20 s has no value here.
    if op in ("ce_fwd", "ce_bwd") and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if op == "rope":
        return {"q": _exact_rope(s["q"], s), "k": _exact_rope(s["k"], s)}
    if op == "muon":
        return _exact_muon(s)
    return _exact_ce(s, op == "ce_bwd")


def _exact_rope(x, s):
    """The pairs as complex numbers times m exp(i t theta)."""
    c, (B, T, _, D) = s["case"], x.shape
    n = c["rot"] // 2
    t = torch.arange(T, device="cuda").repeat(B, 1) if s["positions"] is None else s["positions"]
    phase = torch.einsum("bt,i->bti", t.double(), s["freqs"])
    turn = torch.polar(torch.full_like(phase, s["mscale"]), phase).unsqueeze(2)
    if c["backward"]:
        turn = turn.conj()
    y = x.double()
    if c["interleaved"]:
        z = torch.view_as_complex(y[..., :2 * n].unflatten(-1, (n, 2)).contiguous()) * turn
        y[..., :2 * n] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :n], y[..., n:2 * n]) * turn
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def _exact_ce(s, backward):
    z = torch.einsum("nd,vd->nv", s["x"].double(), s["w"].double())
    t = s["targets"].to(torch.int64)
    has = t >= 0
    rows = torch.arange(t.numel(), device="cuda")
    if not backward:
        zt = z[rows, torch.where(has, t, 0)]
        lse = torch.logsumexp(z, dim=1)
        # ln(1 + sum over the other words of exp(z - zt)), which does not cancel
        z -= zt.unsqueeze(1)
        z[rows, torch.where(has, t, 0)] = -math.inf
        loss = torch.logaddexp(torch.zeros_like(zt), torch.logsumexp(z, dim=1))
        return {"loss": torch.where(has, loss, 0.0), "lse": lse}
    z = torch.exp(z - s["lse"].double()[:, None])
    g = s["dloss"].double() * has
    z = torch.einsum("nv,n->nv", z, g if s["dlse"] is None else g + s["dlse"].double())
    z[rows[has], t[has]] -= g[has]
    return {"dx": torch.einsum("nv,vd->nd", z, s["w"].double()),
            "dw": torch.einsum("nv,nd->vd", z, s["x"].double())}


def _exact_muon(s):
    g, out = s["g"].double(), {}
    if s["momentum"] is not None:
        out["momentum"] = s["momentum"].double() * BETA + g
        g = g + out["momentum"] * BETA
    x = g / (torch.linalg.vector_norm(g, dim=(1, 2), keepdim=True) + EPS)
    a, b, c = NS
    # X is multiplied from the side that is shorter, by (c G + b) G + a with its Gram matrix G.
    wide = _is_wide(s["case"])
    eye = torch.eye(min(x.shape[1:]), dtype=torch.float64, device="cuda")
    for _ in range(NS_STEPS):
        gram = torch.einsum("zik,zjk->zij" if wide else "zki,zkj->zij", x, x)
        p = torch.baddbmm(a * eye.expand_as(gram), c * gram + b * eye, gram)
        x = torch.bmm(p, x) if wide else torch.bmm(x, p)
    out["o"] = x
    return out


def _is_wide(case):
    return case["m"] <= case["n"]
