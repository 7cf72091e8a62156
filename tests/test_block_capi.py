"""Refusals of the block norms, 8-bit checkpoints and gated unit: invalid
arguments return their documented codes before any CUDA call, and the binding
refuses tensors of a wrong kind.  No GPU needed."""
import ctypes

import pytest
import torch

import deterministic_attention_gb300 as da

P = ctypes.c_void_p(0x10000)       # 16-byte aligned stand-in pointer (never dereferenced)
BAD = ctypes.c_void_p(0x10008)     # misaligned
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    da.build()
    return da.lib()


def _ok(rc):
    """Valid: done where there is a GPU (nothing to do), stopped by the missing device here."""
    assert rc in (0, -6)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -3), (dict(d=16), -3), (dict(d=48), -3), (dict(d=(1 << 20) + 32), -3),
    (dict(rows=1 << 30, d=128), -3), (dict(x=None), -1), (dict(q=None), -1), (dict(e=None), -1),
    (dict(x=BAD), -2), (dict(q=BAD), -2)])
def test_pack_and_unpack_reject(L, kw, code):
    a = dict(dict(x=P, q=P, e=P, rows=4, d=64), **kw)
    assert L.act8_pack(a["x"], a["q"], a["e"], a["rows"], a["d"], None) == code
    assert L.act8_unpack(a["q"], a["e"], a["x"], a["rows"], a["d"], None) == code
    assert da.last_error() != ""


def test_empty_checkpoint_is_ok_without_device(L):
    assert L.act8_pack(None, None, None, 0, 32, None) == 0
    assert L.act8_unpack(None, None, None, 0, 32, None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -3), (dict(rows=(1 << 24) + 1), -3), (dict(d=16), -3), (dict(d=40), -3),
    (dict(n=0), -3), (dict(n=12), -3), (dict(rows=1 << 20, n=1 << 20), -3), (dict(q=None), -1),
    (dict(e=None), -1), (dict(dy=None), -1), (dict(dw=None), -1), (dict(q=BAD), -2),
    (dict(dy=BAD), -2), (dict(dw=BAD), -2), (dict(scale=BAD), -2), (dict(ws=None), -9),
    (dict(wsb=64), -9), (dict(ws=BAD), -2)])
def test_wgrad_rejects(L, kw, code):
    a = dict(dict(q=P, e=P, dy=P, scale=None, dw=P, ws=P, wsb=1 << 30, rows=4096, d=768, n=1280), **kw)
    assert L.act8_wgrad(a["q"], a["e"], a["dy"], a["scale"], a["dw"], a["ws"], a["wsb"], a["rows"],
                        a["d"], a["n"], None) == code


def test_wgrad_workspace_follows_the_shape(L):
    tile = 256 * 256 * 4
    assert L.act8_wgrad_workspace_bytes(4096, 768, 1280) == 15 * 5 * tile   # 15 tiles, five ranges each
    assert L.act8_wgrad_workspace_bytes(64, 768, 1280) == 0                 # one step: nothing to cut
    assert L.act8_wgrad_workspace_bytes(4096, 128 * 8, 256 * 19) == 0       # 76 tiles
    assert L.act8_wgrad_workspace_bytes(0, 768, 1280) == 0
    assert L.act8_wgrad_workspace_bytes(4096, 768, 1281) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -3), (dict(f=0), -3), (dict(f=12), -3), (dict(f=40, q=P, e=P), -3),
    (dict(rows=1 << 20, f=1 << 16), -3), (dict(u=None), -1), (dict(h=None), -1), (dict(q=P), -1),
    (dict(e=P), -1), (dict(u=BAD), -2), (dict(h=BAD), -2), (dict(q=BAD, e=P), -2)])
def test_swiglu_fwd_rejects(L, kw, code):
    a = dict(dict(u=P, h=P, q=None, e=None, rows=4, f=64), **kw)
    assert L.swiglu_fwd(a["u"], a["h"], a["q"], a["e"], a["rows"], a["f"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -3), (dict(f=12), -3), (dict(dh=None), -1), (dict(du=None), -1), (dict(u=None), -1),
    (dict(q=P, e=P), -1),                  # u and its checkpoint
    (dict(u=None, q=P), -1), (dict(u=None, q=P, e=P, f=40), -3), (dict(h=BAD), -2), (dict(dh=BAD), -2)])
def test_swiglu_bwd_rejects(L, kw, code):
    a = dict(dict(dh=P, u=P, q=None, e=None, du=P, h=None, rows=4, f=64), **kw)
    assert L.swiglu_bwd(a["dh"], a["u"], a["q"], a["e"], a["du"], a["h"], a["rows"], a["f"], None) == code


FWD = dict(x=P, y=P, gate=P, w_post=P, w_pre=P, x_out=P, h=P, rstd_post=P, rstd_pre=P, yq=None,
           ye=None, xq=None, xe=None, N=8, d=64, G=2, x32=0, g32=1, sig=0, r=1.0, s=1.0, eps=1e-6)


def _fwd(L, **kw):
    return L.block_norm_fwd(*dict(FWD, **kw).values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), -3), (dict(d=0), -3), (dict(d=12), -3), (dict(d=8200), -3), (dict(G=3), -3),
    (dict(G=0), -3), (dict(G=16), -3), (dict(N=1 << 30, d=128), -3),
    (dict(d=40, yq=P, ye=P, xq=P, xe=P), -3), (dict(x32=2), -3), (dict(sig=-1), -3),
    (dict(r=INF), -5), (dict(s=NAN), -5), (dict(eps=0.0), -5), (dict(eps=-1.0), -5), (dict(eps=NAN), -5),
    (dict(x=None), -1), (dict(x_out=None), -1), (dict(h=None), -1), (dict(rstd_pre=None), -1),
    (dict(rstd_post=None), -1), (dict(y=None), -1),      # gate and w_post without a block
    (dict(w_pre=None), -1),                              # h without its weight
    (dict(w_post=None), -1),                             # rstd_post without its norm
    (dict(yq=P), -1), (dict(yq=P, ye=P), -1),            # half a checkpoint; one of the two
    (dict(x=BAD), -2), (dict(gate=BAD), -2), (dict(h=BAD), -2), (dict(yq=BAD, ye=P, xq=P, xe=P), -2),
    (dict(y=None, gate=None, w_post=None, w_pre=None, x_out=None, h=None, rstd_post=None,
          rstd_pre=None), -1)])
def test_block_norm_fwd_rejects(L, kw, code):
    assert _fwd(L, **kw) == code
    assert da.last_error() != ""


def test_block_norm_fwd_valid_forms(L):
    if torch.cuda.is_available():
        pytest.skip("stand-in pointers")
    for kw in (dict(), dict(gate=None), dict(w_post=None, rstd_post=None), dict(ye=BAD, yq=P, xq=P, xe=BAD),
               dict(w_pre=None, h=None, rstd_pre=None), dict(G=8), dict(G=1),
               dict(y=None, gate=None, w_post=None, x_out=None, rstd_post=None)):
        assert _fwd(L, **kw) == -6
    assert _fwd(L, N=0, x=None) == 0


BWD = dict(dx_out=P, dh=P, x=P, y=P, xq=None, xe=None, yq=None, ye=None, gate=P, w_post=P, w_pre=P,
           rstd_post=P, rstd_pre=P, dx=P, dy=P, dgate=P, dw_post=P, dw_pre=P, ws=P, wsb=1 << 30, N=8,
           d=64, G=2, x32=0, g32=1, sig=0, r=1.0, s=1.0)


def _bwd(L, **kw):
    return L.block_norm_bwd(*dict(BWD, **kw).values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), -3), (dict(d=12), -3), (dict(G=3), -3), (dict(x32=3), -3), (dict(g32=-1), -3),
    (dict(r=NAN), -5), (dict(s=INF), -5),
    (dict(dx=None), -1), (dict(dh=None), -1), (dict(x=None), -1), (dict(y=None), -1),
    (dict(rstd_pre=None), -1), (dict(rstd_post=None), -1), (dict(dgate=None), -1),
    (dict(dw_pre=None), -1), (dict(dw_post=None), -1), (dict(dy=None), -1),
    (dict(xq=P, xe=P), -1), (dict(x=None, xq=P, xe=P), -1),   # both kinds; one of each
    (dict(x=None, y=None, xq=P, xe=P, yq=P), -1),
    (dict(y=None, yq=P, ye=P), -1),
    (dict(dx_out=None, dh=None, w_pre=None, x=None, rstd_pre=None, dw_pre=None), -1),
    (dict(dx=BAD), -2), (dict(dy=BAD), -2), (dict(dx_out=BAD), -2), (dict(ws=BAD), -2),
    (dict(ws=None), -9), (dict(wsb=100), -9)])
def test_block_norm_bwd_rejects(L, kw, code):
    assert _bwd(L, **kw) == code
    assert da.last_error() != ""


def test_block_norm_bwd_valid_forms(L):
    if torch.cuda.is_available():
        pytest.skip("stand-in pointers")
    for kw in (dict(), dict(x=None, y=None, xq=P, xe=BAD, yq=P, ye=BAD), dict(dx_out=None),
               dict(gate=None, dgate=None), dict(w_post=None, rstd_post=None, dw_post=None),
               dict(dh=None, x=None, w_pre=None, rstd_pre=None, dw_pre=None),
               dict(gate=None, dgate=None, w_post=None, rstd_post=None, dw_post=None, y=None),
               dict(dy=None, y=None, gate=None, dgate=None, w_post=None, rstd_post=None, dw_post=None)):
        assert _bwd(L, **kw) == -6, (kw, da.last_error())


def test_block_norm_workspace(L):
    up = lambda x: (x + 255) // 256 * 256
    # 4096 rows of 768 columns: eleven rows at a time in each of 152 blocks.
    assert L.block_norm_bwd_workspace_bytes(4096, 768, 1) == 3 * up(152 * 768 * 4)
    assert L.block_norm_bwd_workspace_bytes(0, 768, 1) == 0
    assert L.block_norm_bwd_workspace_bytes(8, 768, 3) == 0
    # A gate row for every two rows: each is one block's, no parts to add up.
    assert L.block_norm_bwd_workspace_bytes(1 << 20, 256, 1 << 19) == 2 * up(152 * 256 * 4)
    # 32 sequences: 19 slices each.
    assert L.block_norm_bwd_workspace_bytes(32768, 1536, 32) == 2 * up(152 * 1536 * 4) + up(608 * 1536 * 4)


def test_binding_refuses_cpu_tensors_and_wrong_kinds(L):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        da.act8_pack(x)
    with pytest.raises(ValueError, match="CUDA"):
        da.swiglu_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        da.block_norm_fwd(x, w_pre=w)
    with pytest.raises(TypeError):
        da.block_norm_fwd([1.0], w_pre=w)
    with pytest.raises(ValueError, match="CUDA"):
        da.act8_wgrad(da.Act8(torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 2), dtype=torch.uint8)), x)
    with pytest.raises(ValueError, match="no gradient"):
        da.block_norm_bwd(None, None, da.BlockNormKept())


def test_statistics_need_four_byte_alignment(L):
    assert _fwd(L, rstd_pre=ctypes.c_void_p(0x10002)) == -2
    assert _bwd(L, rstd_post=ctypes.c_void_p(0x10001)) == -2
    if not torch.cuda.is_available():
        assert _fwd(L, rstd_pre=ctypes.c_void_p(0x10004)) == -6
