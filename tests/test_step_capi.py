"""Refusals of the rotary positions, the output projection's cross entropy and
the orthogonalised update: invalid arguments return their documented codes
before any CUDA call, and the binding refuses tensors of a wrong kind.  No GPU
needed."""
import ctypes

import pytest
import torch

import deterministic_attention_gb300 as da

P = ctypes.c_void_p(0x10000)       # 16-byte aligned stand-in pointer (never dereferenced)
BAD = ctypes.c_void_p(0x10008)     # 8-byte aligned
ODD = ctypes.c_void_p(0x10001)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    da.build()
    return da.lib()


ROPE = dict(q=P, k=P, qo=P, ko=P, f=P, pos=None, n_pos=0, q_ld=256, k_ld=128, qo_ld=256, ko_ld=128, N=6, T=3,
            Hq=4, Hkv=2, D=64, rot=64, inter=0, f32=0, m=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), -3), (dict(N=(1 << 30) + 1), -3), (dict(T=0), -3), (dict(Hq=-1), -3), (dict(Hq=0, Hkv=0), -3),
    (dict(Hq=5000), -3), (dict(D=0), -4), (dict(D=2000), -4), (dict(rot=0), -4), (dict(rot=63), -4),
    (dict(rot=66), -4), (dict(n_pos=-1), -3), (dict(n_pos=3), -3), (dict(pos=P), -3), (dict(q_ld=255), -3),
    (dict(k_ld=100), -3), (dict(qo_ld=8), -3), (dict(ko_ld=-128), -3), (dict(q_ld=512), -3),
    (dict(k_ld=256), -3), (dict(inter=2), -3), (dict(f32=-1), -3), (dict(m=INF), -5), (dict(m=NAN), -5),
    (dict(q=None), -1), (dict(qo=None), -1), (dict(k=None), -1), (dict(ko=None), -1), (dict(f=None), -1),
    (dict(Hkv=0), -1),                      # k without heads
    (dict(q=ODD), -2), (dict(ko=ODD), -2), (dict(f=ctypes.c_void_p(0x10004)), -2),
    (dict(pos=ODD, n_pos=3), -2), (dict(f32=1, q=ctypes.c_void_p(0x10002)), -2)])
def test_rope_rejects(L, kw, code):
    a = dict(ROPE, **kw)
    assert L.rope_fwd(*a.values(), None) == code
    assert da.last_error() != ""
    assert L.rope_bwd(*a.values(), None) == code


def test_rope_valid_forms(L):
    if torch.cuda.is_available():
        pytest.skip("stand-in pointers")
    for kw in (dict(), dict(Hkv=0, k=None, ko=None, k_ld=0, ko_ld=0), dict(pos=P, n_pos=3), dict(q=BAD, rot=2),
               dict(qo=BAD, q_ld=4096)):
        assert L.rope_fwd(*dict(ROPE, **kw).values(), None) == -6
    assert L.rope_fwd(*dict(ROPE, N=0, q=None, f=None).values(), None) == 0


FREQS = dict(rot=64, base=1e4, kind=4, factor=8.0, context=4096, low=1.0, high=4.0)


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), -4), (dict(rot=7), -4), (dict(rot=1026), -4), (dict(kind=5), -3), (dict(kind=-1), -3),
    (dict(base=1.0), -5), (dict(base=INF), -5), (dict(base=NAN), -5), (dict(factor=0.5), -5),
    (dict(factor=NAN), -5), (dict(context=0), -5), (dict(low=0.0), -5), (dict(high=1.0), -5),
    (dict(high=INF), -5), (dict(low=NAN), -5), (dict(kind=2, rot=2), -4)])
def test_rope_freqs_rejects(L, kw, code):
    f, m = (ctypes.c_double * 512)(), ctypes.c_float()
    assert L.rope_freqs(f, ctypes.byref(m), *dict(FREQS, **kw).values()) == code
    assert L.rope_freqs(None, ctypes.byref(m), *FREQS.values()) == -1
    assert L.rope_freqs(f, None, *FREQS.values()) == -1
    assert L.rope_freqs(f, ctypes.byref(m), *FREQS.values()) == 0


CE = dict(x=P, w=P, t=P, loss=P, lse=P, ws=P, wsb=1 << 40, N=300, V=1000, d=64)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), -3), (dict(N=(1 << 24) + 1), -3), (dict(V=0), -3), (dict(V=(1 << 24) + 1), -3),
    (dict(d=0), -3), (dict(d=12), -3), (dict(d=(1 << 16) + 8), -3), (dict(N=1 << 24, d=4096), -3),
    (dict(N=1 << 24, V=1 << 22), -3), (dict(x=None), -1), (dict(w=None), -1), (dict(t=None), -1),
    (dict(loss=None), -1), (dict(lse=None), -1), (dict(x=BAD), -2), (dict(t=BAD), -2), (dict(lse=BAD), -2),
    (dict(ws=None), -9), (dict(wsb=100), -9), (dict(ws=BAD), -2)])
def test_linear_ce_fwd_rejects(L, kw, code):
    assert L.linear_ce_fwd(*dict(CE, **kw).values(), None) == code
    assert da.last_error() != ""


CEB = dict(x=P, w=P, t=P, lse=P, g=P, e=P, dx=P, dw=P, ws=P, wsb=1 << 40, N=300, V=1000, d=64, f32=0)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), -3), (dict(V=0), -3), (dict(d=4), -3), (dict(f32=2), -3), (dict(x=None), -1), (dict(g=None), -1),
    (dict(lse=None), -1), (dict(dx=None), -1), (dict(dw=None), -1), (dict(e=BAD), -2), (dict(dw=BAD), -2),
    (dict(ws=None), -9), (dict(wsb=100), -9), (dict(ws=BAD), -2), (dict(N=0, dw=None), -1)])
def test_linear_ce_bwd_rejects(L, kw, code):
    assert L.linear_ce_bwd(*dict(CEB, **kw).values(), None) == code


def test_linear_ce_sizes(L):
    assert L.linear_ce_fwd(*dict(CE, N=0, x=None).values(), None) == 0
    parts = 2 * 4 * 300 * 8
    assert L.linear_ce_fwd_workspace_bytes(300, 1000, 64) == (parts + 255) // 256 * 256 + 1280
    assert L.linear_ce_fwd_workspace_bytes(0, 1000, 64) == 0
    assert L.linear_ce_bwd_workspace_bytes(300, 1000, 63) == 0
    # A piece of dz is at most 1 GiB, whatever the vocabulary; beyond it come the
    # fp32 sums of dx and partial tiles.
    for N, V in ((4096, 50432), (32768, 50432), (16384, 1 << 20)):
        extra = N * 64 * 4 + 76 * 32 * 256 * 256 * 4
        assert L.linear_ce_bwd_workspace_bytes(N, V, 64) <= (1 << 30) + extra + 4096
    if not torch.cuda.is_available():
        assert L.linear_ce_bwd(*dict(CEB, e=None).values(), None) == -6
        assert L.linear_ce_fwd(*CE.values(), None) == -6


MUON = dict(g=P, m=P, o=P, ws=P, wsb=1 << 40, batch=2, rows=30, cols=64, f32=0, nest=1, steps=5, c=None,
            beta=0.95, eps=1e-7)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -3), (dict(batch=65536), -3), (dict(rows=0), -3), (dict(rows=32769), -3), (dict(cols=0), -3),
    (dict(cols=60), -3), (dict(cols=32776), -3), (dict(batch=1000, rows=8192, cols=8192), -3), (dict(f32=2), -3),
    (dict(nest=-1), -3), (dict(steps=0), -3), (dict(steps=65), -3), (dict(beta=NAN), -5), (dict(eps=0.0), -5),
    (dict(eps=-1.0), -5), (dict(eps=NAN), -5), (dict(eps=INF), -5),
    (dict(steps=1, c=(ctypes.c_float * 3)(1.0, NAN, 0.0)), -5), (dict(g=None), -1), (dict(o=None), -1),
    (dict(g=BAD), -2), (dict(m=BAD), -2), (dict(o=BAD), -2), (dict(ws=None), -9), (dict(wsb=1000), -9),
    (dict(ws=BAD), -2)])
def test_muon_update_rejects(L, kw, code):
    assert L.muon_update(*dict(MUON, **kw).values(), None) == code
    assert da.last_error() != ""


def test_muon_update_valid_forms(L):
    assert L.muon_update(*dict(MUON, batch=0, g=None).values(), None) == 0
    assert L.muon_update_workspace_bytes(0, 30, 64) == 0
    assert L.muon_update_workspace_bytes(2, 30, 63) == 0
    x, s = 2 * 30 * 64 * 2, 2 * 30 * 32 * 2
    up = lambda b: (b + 255) // 256 * 256
    assert L.muon_update_workspace_bytes(2, 30, 64) == 256 + 2 * 3 * 128 + 2 * up(x) + 2 * up(s) + 256
    if not torch.cuda.is_available():
        assert L.muon_update(*dict(MUON, m=None).values(), None) == -6


def test_binding_refuses():
    da.build()
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    f = torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        da.rope_fwd(q, None, f)
    with pytest.raises(TypeError):
        da.rope_fwd(None, q, f)
    with pytest.raises(ValueError, match="scaling"):
        da.rope_freqs(64, scaling="other", device="cpu")
    with pytest.raises(da.DetAttnError):
        da.rope_freqs(63, device="cpu")
    x, w, t = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16), torch.zeros(3)
    with pytest.raises(ValueError, match="CUDA"):
        da.linear_ce_fwd(x, w, t)
    with pytest.raises(ValueError, match="CUDA"):
        da.linear_ce_bwd(x, w, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        da.muon_update(torch.zeros(8, 8))
    with pytest.raises(ValueError, match="m, n"):
        da.muon_update(torch.zeros(8))
    with pytest.raises(TypeError):
        da.muon_update(None)
