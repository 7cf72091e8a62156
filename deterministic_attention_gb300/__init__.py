"""Deterministic causal grouped-query flash attention on sm_103a (GB300).

Thin Python binding over the C-ABI library ``libdetattn.so`` (declared in
``include/detattn.h``).  This module only marshals arguments: every step of
the forward and backward runs in the library's CUDA kernels.  PyTorch is used
for device memory and the current stream.  There is no CPU fallback: if the
library is missing or the device is not sm_103, calls raise.

Layouts: q, o, dout, dq are bf16 [B, T, Hq, D]; k, v, dk, dv are bf16
[B, T, Hkv, D]; lse is fp32 [B, Hq, T] (natural log).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re
from typing import NamedTuple, Optional

import torch

from .build import LIB as _LIB_PATH, build  # noqa: F401

__all__ = ["attn_fwd", "attn_bwd", "attn_bwd_delta", "attn_bwd_dkdv", "attn_bwd_dq",
           "workspace_bytes", "check_status", "set_wait_limit_ns", "selftest_wait_timeout",
           "set_dkdv_split", "set_dkdv_deal", "new_workspace", "rowstats_view", "last_error", "lib",
           "DetAttnError", "STATUS", "header_symbols", "build", "embed_grad",
           "embed_grad_workspace_bytes", "attn_fwd_varlen", "attn_bwd_varlen",
           "varlen_workspace_bytes", "layer_gemm", "layer_workspace_bytes", "LayerState",
           "layer_train_step", "ds_workspace_bytes", "set_bwd_dq_mode", "Act8", "act8_pack",
           "act8_unpack", "act8_wgrad", "act8_wgrad_workspace_bytes", "swiglu_fwd", "swiglu_bwd",
           "BlockNormKept", "BlockNormGrads", "block_norm_fwd", "block_norm_bwd",
           "block_norm_bwd_workspace_bytes"]

STATUS = {0: "DETATTN_OK", -1: "DETATTN_ERR_NULL", -2: "DETATTN_ERR_ALIGN",
          -3: "DETATTN_ERR_SHAPE", -4: "DETATTN_ERR_HEADDIM", -5: "DETATTN_ERR_SCALE",
          -6: "DETATTN_ERR_CUDA", -7: "DETATTN_ERR_DEVICE_TIMEOUT", -8: "DETATTN_ERR_ARCH",
          -9: "DETATTN_ERR_WORKSPACE", -10: "DETATTN_ERR_INDEX"}

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "detattn.h")


class DetAttnError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library with argument types set (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; call deterministic_attention_gb300.build()")
    L = ctypes.CDLL(_LIB_PATH)
    vp, fp, i, f, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.attn_fwd.argtypes = [vp, vp, vp, vp, fp, i, i, i, i, i, f, i, vp]
    L.attn_bwd_workspace_bytes.argtypes = [i, i, i, i, i]
    L.attn_bwd_workspace_bytes.restype = sz
    L.attn_bwd.argtypes = [vp, vp, vp, vp, fp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, f, i, vp]
    L.attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, fp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    L.attn_bwd_noalloc.restype = i
    L.attn_bwd_delta.argtypes = [vp, vp, fp, vp, sz, i, i, i, i, vp]
    L.attn_bwd_dkdv.argtypes = [vp, vp, vp, vp, vp, sz, vp, vp, i, i, i, i, i, f, i, vp]
    L.attn_bwd_dq.argtypes = [vp, vp, vp, vp, vp, sz, vp, i, i, i, i, i, f, i, vp]
    L.attn_fwd_varlen.argtypes = [vp, vp, vp, vp, fp, vp, vp, i, i, i, i, f, i, vp]
    L.attn_fwd_varlen.restype = i
    L.attn_bwd_varlen_workspace_bytes.argtypes = [vp, vp, i, i, i, i]
    L.attn_bwd_varlen_workspace_bytes.restype = sz
    L.attn_bwd_varlen.argtypes = [vp, vp, vp, vp, fp, vp, vp, vp, vp, vp, sz, vp, vp, i, i, i, i, f,
                                  i, vp]
    L.attn_bwd_varlen.restype = i
    L.attn_bwd_ds_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.attn_bwd_ds_workspace_bytes.restype = sz
    L.detattn_set_bwd_dq_mode.argtypes = [i]
    L.detattn_set_bwd_dq_mode.restype = i
    L.layer_gemm.argtypes = [vp, i, i, vp, i, i, vp, i, i, i, i, i, f, vp]
    L.layer_gemm.restype = i
    L.layer_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.layer_workspace_bytes.restype = sz
    L.layer_train_step.argtypes = [vp] * 15 + [sz] + [i] * 7 + [f] * 5 + [vp]
    L.layer_train_step.restype = i
    L.embed_grad_workspace_bytes.argtypes = [i, i, i]
    L.embed_grad_workspace_bytes.restype = sz
    L.embed_grad.argtypes = [vp, vp, vp, vp, sz, i, i, i, vp]
    L.embed_grad.restype = i
    L.act8_pack.argtypes = [vp, vp, vp, i, i, vp]
    L.act8_unpack.argtypes = [vp, vp, vp, i, i, vp]
    L.act8_wgrad_workspace_bytes.argtypes = [i, i, i]
    L.act8_wgrad_workspace_bytes.restype = sz
    L.act8_wgrad.argtypes = [vp] * 6 + [sz, i, i, i, vp]
    L.swiglu_fwd.argtypes = [vp, vp, vp, vp, i, i, vp]
    L.swiglu_bwd.argtypes = [vp] * 6 + [i, i, vp]
    L.block_norm_fwd.argtypes = [vp] * 13 + [i] * 6 + [f] * 3 + [vp]
    L.block_norm_bwd_workspace_bytes.argtypes = [i, i, i]
    L.block_norm_bwd_workspace_bytes.restype = sz
    L.block_norm_bwd.argtypes = [vp] * 19 + [sz] + [i] * 6 + [f] * 2 + [vp]
    for name in ("act8_pack", "act8_unpack", "act8_wgrad", "swiglu_fwd", "swiglu_bwd",
                 "block_norm_fwd", "block_norm_bwd"):
        getattr(L, name).restype = i
    L.detattn_check_status.argtypes = [vp]
    L.detattn_diag_exp2.argtypes = [vp, vp, vp, vp, i, vp]
    L.detattn_diag_exp2.restype = i
    L.detattn_diag_qtile_deal.argtypes = [i, i, i, i, i, i, vp, i]
    L.detattn_diag_qtile_deal.restype = i
    L.detattn_diag_dkdv_split.argtypes = [i, i, i, i, i, i, vp, i, vp, vp]
    L.detattn_diag_dkdv_split.restype = i
    L.detattn_selftest_wait_timeout.argtypes = [ctypes.c_ulonglong, vp]
    L.detattn_selftest_wait_timeout.restype = i
    L.detattn_set_dkdv_split.argtypes = [i]
    L.detattn_set_dkdv_split.restype = i
    L.detattn_diag_dkdv_list.argtypes = [i, i, i, i, i, i, i, i, vp, vp, i]
    L.detattn_diag_dkdv_list.restype = i
    L.detattn_set_dkdv_deal.argtypes = [i]
    L.detattn_set_dkdv_deal.restype = i
    L.detattn_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    L.detattn_set_wait_limit_ns.restype = None
    L.detattn_last_error.argtypes = []
    L.detattn_last_error.restype = ctypes.c_char_p
    L.detattn_version.argtypes = []
    for name in ("attn_fwd", "attn_bwd", "attn_bwd_delta", "attn_bwd_dkdv", "attn_bwd_dq",
                 "detattn_check_status", "detattn_version"):
        getattr(L, name).restype = i
    _lib = L
    return L


def header_symbols() -> list[str]:
    """Function names declared in include/detattn.h."""
    text = open(HEADER).read()
    return re.findall(r"^\s*(?:int|size_t|void|const char\*)\s+(\w+)\s*\(", text, re.M)


def last_error() -> str:
    return lib().detattn_last_error().decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise DetAttnError(rc, where, last_error())


def _stream():
    # The raw handle of the current device's current stream: 0.2 us, against
    # 2.9 us for building the torch.cuda.Stream object around it.
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, name, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be 4-D [B, T, H, D]")
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    return B, T, Hq, Hkv, D


def _scale(scale, D):
    return float(1.0 / math.sqrt(D) if scale is None else scale)


def attn_fwd(q, k, v, scale=None, causal=True, out=None, lse=None):
    """Forward: returns (o bf16 [B,T,Hq,D], lse fp32 [B,Hq,T])."""
    B, T, Hq, Hkv, D = _dims(q, k)
    bf = torch.bfloat16
    _need(q, "q", bf, (B, T, Hq, D))
    _need(k, "k", bf, (B, T, Hkv, D))
    _need(v, "v", bf, (B, T, Hkv, D))
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(o, "o", bf, (B, T, Hq, D))
    _need(l, "lse", torch.float32, (B, Hq, T))
    rc = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, T, Hq, Hkv, D,
                        _scale(scale, D), int(bool(causal)), _stream())
    _check(rc, "attn_fwd")
    return o, l


def workspace_bytes(B, T, Hq, Hkv, D) -> int:
    return int(lib().attn_bwd_workspace_bytes(B, T, Hq, Hkv, D))


def attn_bwd(q, k, v, o, lse, dout, scale=None, causal=True, dq=None, dk=None, dv=None,
             workspace=None):
    """Backward: returns (dq, dk, dv), bf16, in the layouts of q, k, v."""
    B, T, Hq, Hkv, D = _dims(q, k)
    bf = torch.bfloat16
    for t, n, s in ((q, "q", (B, T, Hq, D)), (k, "k", (B, T, Hkv, D)), (v, "v", (B, T, Hkv, D)),
                    (o, "o", (B, T, Hq, D)), (dout, "dout", (B, T, Hq, D))):
        _need(t, n, bf, s)
    _need(lse, "lse", torch.float32, (B, Hq, T))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _need(dq, "dq", bf, (B, T, Hq, D))
    _need(dk, "dk", bf, (B, T, Hkv, D))
    _need(dv, "dv", bf, (B, T, Hkv, D))
    if workspace is None:
        workspace = new_workspace(B, T, Hq, Hkv, D, q.device)
    rc = lib().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                        _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(), B, T, Hq, Hkv, D,
                        _scale(scale, D), int(bool(causal)), _stream())
    _check(rc, "attn_bwd")
    return dq, dk, dv


def ds_workspace_bytes(B, T, Hq, Hkv, D, causal=True) -> int:
    return int(lib().attn_bwd_ds_workspace_bytes(B, T, Hq, Hkv, D, int(bool(causal))))


def new_workspace(B, T, Hq, Hkv, D, device="cuda", stored_ds=False, causal=True):
    """A device workspace (uint8) of attn_bwd_workspace_bytes, or with
    stored_ds of attn_bwd_ds_workspace_bytes (the stored-dS backward)."""
    n = ds_workspace_bytes(B, T, Hq, Hkv, D, causal) if stored_ds else 0
    if n == 0:
        n = workspace_bytes(B, T, Hq, Hkv, D)
    return torch.empty((max(16, n),), dtype=torch.uint8, device=device)


def set_bwd_dq_mode(mode: int):
    """0 (default): the dQ step recomputes S and dP; 1: stored-dS backward
    whenever the workspace holds it (new_workspace(..., stored_ds=True))."""
    _check(lib().detattn_set_bwd_dq_mode(int(mode)), "detattn_set_bwd_dq_mode")


def rowstats_view(workspace, B, T, Hq):
    """The workspace's row statistics as fp32 [B, Hq, Tp, 2]:
    [..., 0] = -LSE*log2(e), [..., 1] = -Delta (see include/detattn.h)."""
    Tp = (T + 127) // 128 * 128
    return workspace[: B * Hq * Tp * 8].view(torch.float32).view(B, Hq, Tp, 2)


def attn_bwd_delta(o, dout, lse, workspace):
    """Backward step 1: row statistics (from o, dout, lse) into `workspace`."""
    B, T, Hq, D = o.shape
    _need(o, "o", torch.bfloat16, (B, T, Hq, D))
    _need(dout, "dout", torch.bfloat16, (B, T, Hq, D))
    _need(lse, "lse", torch.float32, (B, Hq, T))
    _check(lib().attn_bwd_delta(_ptr(o), _ptr(dout), _ptr(lse), _ptr(workspace), workspace.numel(),
                                B, T, Hq, D, _stream()), "attn_bwd_delta")
    return workspace


def attn_bwd_dkdv(q, k, v, dout, workspace, scale=None, causal=True, dk=None, dv=None):
    """Backward step 2: dk, dv from the row statistics in `workspace`."""
    B, T, Hq, Hkv, D = _dims(q, k)
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(lib().attn_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(workspace),
                               workspace.numel(), _ptr(dk), _ptr(dv), B, T, Hq, Hkv, D,
                               _scale(scale, D), int(bool(causal)), _stream()), "attn_bwd_dkdv")
    return dk, dv


def attn_bwd_dq(q, k, v, dout, workspace, scale=None, causal=True, dq=None):
    """Backward step 3: dq from the row statistics in `workspace`."""
    B, T, Hq, Hkv, D = _dims(q, k)
    dq = torch.empty_like(q) if dq is None else dq
    _check(lib().attn_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(workspace),
                             workspace.numel(), _ptr(dq), B, T, Hq, Hkv, D, _scale(scale, D),
                             int(bool(causal)), _stream()), "attn_bwd_dq")
    return dq


def _host_cu(cu):
    """Offsets as a contiguous host int32 array (kept alive by the caller)."""
    import numpy as np
    if isinstance(cu, torch.Tensor):
        cu = cu.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(cu, dtype=np.int32).reshape(-1))


def varlen_workspace_bytes(cu_q, cu_k, Hq, Hkv, D) -> int:
    cq, ck = _host_cu(cu_q), _host_cu(cu_k)
    return int(lib().attn_bwd_varlen_workspace_bytes(ctypes.c_void_p(cq.ctypes.data),
                                                     ctypes.c_void_p(ck.ctypes.data),
                                                     cq.size - 1, Hq, Hkv, D))


def attn_fwd_varlen(q, k, v, cu_q, cu_k, scale=None, causal=True, out=None, lse=None):
    """Packed variable-length forward: q [total_q, Hq, D], k, v [total_k, Hkv,
    D]; sequence s is query rows cu_q[s]..cu_q[s+1]-1 and key rows
    cu_k[s]..cu_k[s+1]-1 (cu_q, cu_k on the host).  Returns o [total_q, Hq,
    D] and lse fp32 [Hq, total_q] (-inf for rows that see no key)."""
    Nq, Hq, D = q.shape
    Nk, Hkv = k.shape[0], k.shape[1]
    bf = torch.bfloat16
    _need(q, "q", bf, (Nq, Hq, D))
    _need(k, "k", bf, (Nk, Hkv, D))
    _need(v, "v", bf, (Nk, Hkv, D))
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(o, "o", bf, (Nq, Hq, D))
    _need(l, "lse", torch.float32, (Hq, Nq))
    cq, ck = _host_cu(cu_q), _host_cu(cu_k)
    rc = lib().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l),
                               ctypes.c_void_p(cq.ctypes.data), ctypes.c_void_p(ck.ctypes.data),
                               cq.size - 1, Hq, Hkv, D, _scale(scale, D), int(bool(causal)),
                               _stream())
    _check(rc, "attn_fwd_varlen")
    return o, l


def attn_bwd_varlen(q, k, v, o, lse, dout, cu_q, cu_k, scale=None, causal=True, dq=None,
                    dk=None, dv=None, workspace=None):
    """Packed variable-length backward: (dq, dk, dv) in the layouts of q, k, v."""
    Nq, Hq, D = q.shape
    Nk, Hkv = k.shape[0], k.shape[1]
    bf = torch.bfloat16
    for t, n, shp in ((q, "q", (Nq, Hq, D)), (k, "k", (Nk, Hkv, D)), (v, "v", (Nk, Hkv, D)),
                      (o, "o", (Nq, Hq, D)), (dout, "dout", (Nq, Hq, D))):
        _need(t, n, bf, shp)
    _need(lse, "lse", torch.float32, (Hq, Nq))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    cq, ck = _host_cu(cu_q), _host_cu(cu_k)
    if workspace is None:
        workspace = torch.empty((max(16, varlen_workspace_bytes(cq, ck, Hq, Hkv, D)),),
                                dtype=torch.uint8, device=q.device)
    rc = lib().attn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                               _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(),
                               ctypes.c_void_p(cq.ctypes.data), ctypes.c_void_p(ck.ctypes.data),
                               cq.size - 1, Hq, Hkv, D, _scale(scale, D), int(bool(causal)),
                               _stream())
    _check(rc, "attn_bwd_varlen")
    return dq, dk, dv


def layer_gemm(a, b, a_mn_major=False, b_mn_major=True, out=None, out_fp32=False, alpha=1.0):
    """C = alpha A B on the tensor cores (bf16 in, fp32 accumulation).  a is
    [M, K] (or, with a_mn_major, stored transposed as [K, M]); b is [K, N]
    with b_mn_major (the default, row-major B) or stored transposed [N, K]."""
    M, K = (a.shape[1], a.shape[0]) if a_mn_major else tuple(a.shape)
    N = b.shape[1] if b_mn_major else b.shape[0]
    if (b.shape[0] if b_mn_major else b.shape[1]) != K:
        raise ValueError(f"inner dimensions differ: a {tuple(a.shape)}, b {tuple(b.shape)}")
    _need(a, "a", torch.bfloat16, tuple(a.shape))
    _need(b, "b", torch.bfloat16, tuple(b.shape))
    dt = torch.float32 if out_fp32 else torch.bfloat16
    c = torch.empty((M, N), dtype=dt, device=a.device) if out is None else out
    _need(c, "c", dt, (M, N))
    _check(lib().layer_gemm(_ptr(a), int(a_mn_major), a.shape[1], _ptr(b), int(b_mn_major),
                            b.shape[1], _ptr(c), int(out_fp32), N, M, N, K, float(alpha),
                            _stream()), "layer_gemm")
    return c


def layer_workspace_bytes(B, T, d, Hq, Hkv, D) -> int:
    return int(lib().layer_workspace_bytes(B, T, d, Hq, Hkv, D))


class LayerState:
    """Device state of one attention layer under AdamW: fp32 master weights
    w_qkv [d, (Hq + 2 Hkv) D] (= [Wq | Wk | Wv]) and w_o [Hq D, d], their
    moments, bf16 copies, gradient buffers and the step workspace."""

    def __init__(self, wq, wk, wv, wo, B, T, Hq, Hkv, D, device="cuda"):
        d = wq.shape[0]
        self.dims = (B, T, d, Hq, Hkv, D)
        f32 = dict(dtype=torch.float32, device=device)
        self.w_qkv = torch.cat([wq, wk, wv], dim=1).to(**f32).contiguous()
        self.w_o = wo.to(**f32).contiguous()
        self.m_qkv, self.v_qkv = torch.zeros_like(self.w_qkv), torch.zeros_like(self.w_qkv)
        self.m_o, self.v_o = torch.zeros_like(self.w_o), torch.zeros_like(self.w_o)
        self.w_qkv_bf16 = self.w_qkv.to(torch.bfloat16)
        self.w_o_bf16 = self.w_o.to(torch.bfloat16)
        self.g_qkv, self.g_o = torch.empty_like(self.w_qkv), torch.empty_like(self.w_o)
        self.y = torch.empty((B, T, d), dtype=torch.bfloat16, device=device)
        self.dx = torch.empty((B, T, d), dtype=torch.bfloat16, device=device)
        self.workspace = torch.empty((layer_workspace_bytes(*self.dims),), dtype=torch.uint8,
                                     device=device)
        self.step = 0


def layer_train_step(state, x, dy, lr=3e-4, weight_decay=0.1, beta1=0.9, beta2=0.999, eps=1e-8,
                     with_dx=True):
    """One training step of the layer on (x, dy), then AdamW; returns
    (g_qkv, g_o) of this step (the state's buffers)."""
    B, T, d, Hq, Hkv, D = state.dims
    _need(x, "x", torch.bfloat16, (B, T, d))
    _need(dy, "dy", torch.bfloat16, (B, T, d))
    state.step += 1
    s = state
    _check(lib().layer_train_step(_ptr(x), _ptr(dy), _ptr(s.w_qkv), _ptr(s.w_o), _ptr(s.m_qkv),
                                  _ptr(s.v_qkv), _ptr(s.m_o), _ptr(s.v_o), _ptr(s.w_qkv_bf16),
                                  _ptr(s.w_o_bf16), _ptr(s.g_qkv), _ptr(s.g_o), _ptr(s.y),
                                  _ptr(s.dx) if with_dx else None, _ptr(s.workspace),
                                  s.workspace.numel(), B, T, d, Hq, Hkv, D, s.step, float(lr),
                                  float(weight_decay), float(beta1), float(beta2), float(eps),
                                  _stream()), "layer_train_step")
    return s.g_qkv, s.g_o


# ------------------------------------------------------------ block norms, 8-bit checkpoints
class Act8(NamedTuple):
    """An 8-bit checkpoint of a [rows, d] activation (include/detattn.h):
    q int8 [rows, d], e uint8 [rows, d / 32]; the values are q 2^(e - 127)."""
    q: torch.Tensor
    e: torch.Tensor


class BlockNormKept(NamedTuple):
    """What block_norm_bwd needs of a forward: the row statistics, and either
    the tensors x (x', the stream after the block) and y, or the 8-bit
    checkpoints of the normed x' and y."""
    rstd_pre: Optional[torch.Tensor] = None
    rstd_post: Optional[torch.Tensor] = None
    x: Optional[torch.Tensor] = None
    y: Optional[torch.Tensor] = None
    xhat8: Optional[Act8] = None
    yhat8: Optional[Act8] = None


class BlockNormGrads(NamedTuple):
    dx: torch.Tensor
    dy: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]


def _on_device(t, name, dtype, shape, dev):
    """_need, on the device with index `dev`; one test where all is well."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _addr(t):
    return None if t is None else t.data_ptr()


def _rows(t, name):
    """(rows, d) of a [..., d] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() < 1 or t.shape[-1] == 0:
        raise ValueError(f"{name} must be [..., d] with d >= 1")
    d = t.shape[-1]
    return t.numel() // d, d


def _current(t, name):
    """The current device's index; what is on the CPU has none.  (The calls run
    on the current device's current stream; a tensor of another device is
    refused by _on_device.)"""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path)")
    return torch._C._cuda_getDevice()


def _need_act8(c, name, shape, dev):
    if not isinstance(c, tuple) or len(c) != 2:
        raise TypeError(f"{name} must be an Act8 (q, e)")
    _on_device(c[0], name + ".q", torch.int8, shape, dev)
    _on_device(c[1], name + ".e", torch.uint8, shape[:-1] + (shape[-1] // 32,), dev)


def _new_act8(shape, device):
    if shape[-1] % 32:
        raise ValueError(f"an 8-bit checkpoint needs a multiple of 32 columns, got {shape[-1]}")
    return Act8(torch.empty(shape, dtype=torch.int8, device=device),
                torch.empty(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8, device=device))


def act8_pack(x, out=None):
    """The 8-bit checkpoint of x, bf16 [..., d], d a multiple of 32."""
    rows, d = _rows(x, "x")
    dev = _current(x, "x")
    _on_device(x, "x", torch.bfloat16, x.shape, dev)
    c = out
    if c is None:
        c = _new_act8(x.shape, x.device)
    else:
        _need_act8(c, "out", x.shape, dev)
    _check(lib().act8_pack(x.data_ptr(), c[0].data_ptr(), c[1].data_ptr(), rows, d, _stream()),
           "act8_pack")
    return c


def act8_unpack(c, out=None):
    """The values of an 8-bit checkpoint, bf16 [..., d] (exact)."""
    q, e = c
    rows, d = _rows(q, "q")
    dev = _current(q, "q")
    _need_act8(c, "checkpoint", q.shape, dev)
    x = out
    if x is None:
        x = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    else:
        _on_device(x, "out", torch.bfloat16, q.shape, dev)
    _check(lib().act8_unpack(q.data_ptr(), e.data_ptr(), x.data_ptr(), rows, d, _stream()),
           "act8_unpack")
    return x


@functools.lru_cache(maxsize=256)
def act8_wgrad_workspace_bytes(rows, d, n) -> int:
    return int(lib().act8_wgrad_workspace_bytes(rows, d, n))


def act8_wgrad(c, dy, row_scale=None, dw=None, workspace=None):
    """Weight gradient dw fp32 [d, n] = diag(row_scale) x^T dy from the 8-bit
    checkpoint of the layer input x [..., d] and dy bf16 [..., n]."""
    q, e = c
    rows, d = _rows(q, "q")
    rows_dy, n = _rows(dy, "dy")
    dev = _current(dy, "dy")
    _need_act8(c, "checkpoint", q.shape, dev)
    _on_device(dy, "dy", torch.bfloat16, dy.shape, dev)
    if rows != rows_dy:
        raise ValueError(f"the checkpoint has {rows} rows, dy {rows_dy}")
    if row_scale is not None:
        _on_device(row_scale, "row_scale", torch.float32, (d,), dev)
    if dw is None:
        dw = torch.empty((d, n), dtype=torch.float32, device=dy.device)
    else:
        _on_device(dw, "dw", torch.float32, (d, n), dev)
    size = 0
    if workspace is None:
        size = act8_wgrad_workspace_bytes(rows, d, n)
        if size:
            workspace = torch.empty((size,), dtype=torch.uint8, device=dy.device)
    else:
        size = _workspace_size(workspace, dev)
    _check(lib().act8_wgrad(q.data_ptr(), e.data_ptr(), dy.data_ptr(), _addr(row_scale),
                            dw.data_ptr(), _addr(workspace), size, rows, d, n, _stream()),
           "act8_wgrad")
    return dw


def _workspace_size(w, dev):
    _on_device(w, "workspace", torch.uint8, (w.numel(),), dev)
    return w.numel()


def swiglu_fwd(u, keep8=False, out=None):
    """h = a sigma(a) b for u = [a | b], bf16 [..., 2 f]; with keep8 returns
    (h, the 8-bit checkpoint of u)."""
    rows, f2 = _rows(u, "u")
    dev = _current(u, "u")
    _on_device(u, "u", torch.bfloat16, u.shape, dev)
    if f2 % 2:
        raise ValueError(f"u has {f2} columns, needs 2 f")
    f = f2 // 2
    if keep8 and f % 32:
        raise ValueError(f"an 8-bit checkpoint of u needs f a multiple of 32, got {f}")
    shape = u.shape[:-1] + (f,)
    h = out
    if h is None:
        h = torch.empty(shape, dtype=torch.bfloat16, device=u.device)
    else:
        _on_device(h, "out", torch.bfloat16, shape, dev)
    c = _new_act8(u.shape, u.device) if keep8 else (None, None)
    _check(lib().swiglu_fwd(u.data_ptr(), h.data_ptr(), _addr(c[0]), _addr(c[1]), rows, f,
                            _stream()), "swiglu_fwd")
    return (h, c) if keep8 else h


def swiglu_bwd(dh, u, with_h=False, du=None):
    """du bf16 [..., 2 f] from dh [..., f] and u, bf16 [..., 2 f] or its 8-bit
    checkpoint; with_h: (du, h), h recomputed from the same u."""
    rows, f = _rows(dh, "dh")
    dev = _current(dh, "dh")
    _on_device(dh, "dh", torch.bfloat16, dh.shape, dev)
    shape = dh.shape[:-1] + (2 * f,)
    q = e = None
    if isinstance(u, torch.Tensor):
        _on_device(u, "u", torch.bfloat16, shape, dev)
    else:
        _need_act8(u, "u", shape, dev)
        (q, e), u = u, None
    if du is None:
        du = torch.empty(shape, dtype=torch.bfloat16, device=dh.device)
    else:
        _on_device(du, "du", torch.bfloat16, shape, dev)
    h = torch.empty(dh.shape, dtype=torch.bfloat16, device=dh.device) if with_h else None
    _check(lib().swiglu_bwd(dh.data_ptr(), _addr(u), _addr(q), _addr(e), du.data_ptr(), _addr(h),
                            rows, f, _stream()), "swiglu_bwd")
    return (du, h) if with_h else du


def _need_stream(x, name, shape, dev):
    """A tensor of the residual stream's kind: bf16 or fp32."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not torch.bfloat16 and x.dtype is not torch.float32:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {x.dtype}")
    _on_device(x, name, x.dtype, shape, dev)


def _gate_rows(gate, rows, d, dev):
    """G of a gate [d], [..., d] whose rows divide the stream's."""
    g, dg = _rows(gate, "gate")
    _need_stream(gate, "gate", gate.shape, dev)
    if dg != d or g < 1 or (rows and (g > rows or rows % g)):
        raise ValueError(f"gate has shape {tuple(gate.shape)}: needs d = {d} columns and a number "
                         f"of rows that divides {rows}")
    return g


def block_norm_fwd(x, y=None, gate=None, w_post=None, w_pre=None, res_scale=1.0, block_scale=1.0,
                   eps=1e-6, gate_sigmoid=False, keep8=False, x_out=None):
    """x' = res_scale x + block_scale g norm(y) w_post, h = norm(x') w_pre
    (include/detattn.h): returns (x', h, kept).  x [..., d] is the residual
    stream (bf16 or fp32), y bf16 the block's output (None: x' is x), gate
    [d] or [..., d] (its sigmoid with gate_sigmoid): G rows in all, each shared
    by N / G consecutive rows of the stream, so [d] is one for every channel,
    [B, d] one for each sequence of a [B, T, d] stream and [B, T, d] one for
    each token (a [T, d] gate is not repeated over B).  w_post and w_pre fp32 [d] or None.  kept is what
    block_norm_bwd takes: the row statistics with x' and y, or, with keep8,
    with their normed values in 8 bits."""
    rows, d = _rows(x, "x")
    device = x.device
    dev = _current(x, "x")
    shape, f32, bf = x.shape, torch.float32, torch.bfloat16
    _need_stream(x, "x", shape, dev)
    G, out = 1, x
    if y is not None:
        _on_device(y, "y", bf, shape, dev)
        if gate is not None:
            G = _gate_rows(gate, rows, d, dev)
        if x_out is None:
            out = torch.empty_like(x)
        else:
            out = x_out
            _on_device(out, "x_out", x.dtype, shape, dev)
    elif gate is not None or w_post is not None or x_out is not None:
        raise ValueError("gate, w_post and x_out belong to a block output y")
    h = rp = ro = None
    if w_pre is not None:
        _on_device(w_pre, "w_pre", f32, (d,), dev)
        h = torch.empty(shape, dtype=bf, device=device)
        rp = torch.empty(shape[:-1], dtype=f32, device=device)
    if w_post is not None:
        _on_device(w_post, "w_post", f32, (d,), dev)
        ro = torch.empty(shape[:-1], dtype=f32, device=device)
    xq = xe = yq = ye = None
    if keep8:
        if w_pre is not None:
            xq, xe = _new_act8(shape, device)
        if y is not None:
            yq, ye = _new_act8(shape, device)
    _check(lib().block_norm_fwd(
        x.data_ptr(), _addr(y), _addr(gate), _addr(w_post), _addr(w_pre),
        None if y is None else out.data_ptr(), _addr(h), _addr(ro), _addr(rp), _addr(yq), _addr(ye),
        _addr(xq), _addr(xe), rows, d, G, x.dtype is f32, gate is not None and gate.dtype is f32,
        bool(gate_sigmoid), res_scale, block_scale, eps, _stream()), "block_norm_fwd")
    if keep8:
        return out, h, BlockNormKept(rp, ro, None, None, None if xq is None else Act8(xq, xe),
                                     None if yq is None else Act8(yq, ye))
    return out, h, BlockNormKept(rp, ro, out, y)


@functools.lru_cache(maxsize=256)
def block_norm_bwd_workspace_bytes(N, d, G=1) -> int:
    return int(lib().block_norm_bwd_workspace_bytes(N, d, G))


def block_norm_bwd(dx_out, dh, kept, gate=None, w_post=None, w_pre=None, res_scale=1.0,
                   block_scale=1.0, gate_sigmoid=False, has_block=None, dx=None, workspace=None):
    """Gradients (dx, dy, dgate, dw_post, dw_pre) of block_norm_fwd from dx_out,
    the gradient of x' (None: zero; then the stream is bf16 unless kept.x says
    otherwise), dh, the gradient of h (None with w_pre None), and what the
    forward kept.  has_block: whether the forward had a y (None: whether kept
    holds y or its checkpoint)."""
    like, name = (dx_out, "dx_out") if dx_out is not None else (dh, "dh")
    if like is None:
        raise ValueError("dx_out and dh are both None: no gradient to carry back")
    rows, d = _rows(like, name)
    device = like.device
    dev = _current(like, name)
    shape, f32, bf = like.shape, torch.float32, torch.bfloat16
    rstd_pre, rstd_post, kx, ky, x8, y8 = kept
    block = (ky is not None or y8 is not None) if has_block is None else bool(has_block)
    if (w_pre is None) != (dh is None):
        raise ValueError("dh and w_pre go together")
    if not block and (w_post is not None or gate is not None):
        raise ValueError("gate and w_post belong to a block output y")
    stream = bf
    if dx_out is not None:
        _need_stream(dx_out, "dx_out", shape, dev)
        stream = dx_out.dtype
    elif kx is not None:
        _need_stream(kx, "kept.x", shape, dev)
        stream = kx.dtype
    x = y = xq = xe = yq = ye = rp = ro = dy = dgate = dwo = dwp = None
    if w_pre is not None:
        _on_device(dh, "dh", bf, shape, dev)
        _on_device(w_pre, "w_pre", f32, (d,), dev)
        rp = rstd_pre
        _on_device(rp, "kept.rstd_pre", f32, shape[:-1], dev)
        if x8 is not None:
            _need_act8(x8, "kept.xhat8", shape, dev)
            xq, xe = x8
        else:
            x = kx
            _on_device(x, "kept.x", stream, shape, dev)
        dwp = torch.empty_like(w_pre)
    if w_post is not None:
        _on_device(w_post, "w_post", f32, (d,), dev)
        ro = rstd_post
        _on_device(ro, "kept.rstd_post", f32, shape[:-1], dev)
        dwo = torch.empty_like(w_post)
    G = 1
    if gate is not None:
        G = _gate_rows(gate, rows, d, dev)
        dgate = torch.empty_like(gate)
    if w_post is not None or gate is not None:
        if y8 is not None:
            _need_act8(y8, "kept.yhat8", shape, dev)
            yq, ye = y8
        else:
            y = ky
            _on_device(y, "kept.y", bf, shape, dev)
    if dx is None:
        dx = torch.empty(shape, dtype=stream, device=device)
    else:
        _on_device(dx, "dx", stream, shape, dev)
    if block:
        dy = torch.empty(shape, dtype=bf, device=device)
    if workspace is None:
        size = max(16, block_norm_bwd_workspace_bytes(rows, d, G))
        workspace = torch.empty((size,), dtype=torch.uint8, device=device)
    else:
        size = _workspace_size(workspace, dev)
    _check(lib().block_norm_bwd(
        _addr(dx_out), _addr(dh), _addr(x), _addr(y), _addr(xq), _addr(xe), _addr(yq), _addr(ye),
        _addr(gate), _addr(w_post), _addr(w_pre), _addr(ro), _addr(rp), dx.data_ptr(), _addr(dy),
        _addr(dgate), _addr(dwo), _addr(dwp), workspace.data_ptr(), size, rows, d, G, stream is f32,
        gate is not None and gate.dtype is f32, bool(gate_sigmoid), res_scale, block_scale,
        _stream()), "block_norm_bwd")
    return BlockNormGrads(dx, dy, dgate, dwo, dwp)


def embed_grad_workspace_bytes(N, V, E) -> int:
    return int(lib().embed_grad_workspace_bytes(N, V, E))


def embed_grad(ids, dy, V, dw=None, workspace=None):
    """Deterministic embedding-lookup gradient: dw fp32 [V, E] with
    dw[v] = sum of dy[t] over tokens t with ids[t] == v (include/detattn.h)."""
    if ids.dim() != 1 or dy.dim() != 2:
        raise ValueError("ids must be [N] and dy [N, E]")
    N, E = dy.shape
    _need(ids, "ids", torch.int32, (N,))
    _need(dy, "dy", torch.bfloat16, (N, E))
    dw = torch.empty((V, E), dtype=torch.float32, device=dy.device) if dw is None else dw
    _need(dw, "dw", torch.float32, (V, E))
    if workspace is None:
        workspace = torch.empty((max(16, embed_grad_workspace_bytes(N, V, E)),), dtype=torch.uint8,
                                device=dy.device)
    _check(lib().embed_grad(_ptr(ids), _ptr(dy), _ptr(dw), _ptr(workspace), workspace.numel(), N,
                            V, E, _stream()), "embed_grad")
    return dw


def check_status():
    """Synchronises the current stream and raises if a kernel timed out."""
    _check(lib().detattn_check_status(_stream()), "detattn_check_status")


def diag_qtile_deal(D, B, T, Hq, causal, sms):
    """(number of pipelines, numpy int32 pipeline of each unit) of the static
    query-tile deal; host-only, no GPU needed."""
    import numpy as np
    n = B * Hq * -(-T // 128) if B > 0 and T > 0 else 0
    out = np.empty(max(1, n), dtype=np.int32)
    rc = lib().detattn_diag_qtile_deal(D, B, T, Hq, int(bool(causal)), sms,
                                       ctypes.c_void_p(out.ctypes.data), n)
    if rc < 0:
        raise DetAttnError(rc, "detattn_diag_qtile_deal", last_error())
    return rc, out[:n]


def diag_dkdv_split(B, T, Hq, Hkv, D, causal, resident, blocks_per_key_tile=0):
    """(C, NG) the dK/dV step would choose on a device holding resident[i]
    clusters of 2**i blocks (i = 0..3); host-only, no GPU needed."""
    import numpy as np
    res = np.zeros(4, dtype=np.int32)
    res[:len(resident)] = resident
    c, ng = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().detattn_diag_dkdv_split(B, T, Hq, Hkv, D, int(bool(causal)),
                                       ctypes.c_void_p(res.ctypes.data), blocks_per_key_tile,
                                       ctypes.byref(c), ctypes.byref(ng))
    if rc < 0:
        raise DetAttnError(rc, "detattn_diag_dkdv_split", last_error())
    return c.value, ng.value


def diag_dkdv_list(B, T, Hq, Hkv, causal, c, ng, force=False):
    """The listed deal of the 64-dim dK/dV step's key tiles over ng clusters
    of c blocks: a list, per block, of (tile, shared) pairs, or None where
    the plain walk is used (see include/detattn.h); host-only."""
    import numpy as np
    nb = ng * c
    start = np.zeros(nb + 1, dtype=np.int32)
    cap = 4096
    entry = np.zeros(cap, dtype=np.int32)
    rc = lib().detattn_diag_dkdv_list(B, T, Hq, Hkv, int(bool(causal)), c, ng, int(bool(force)),
                                      ctypes.c_void_p(start.ctypes.data),
                                      ctypes.c_void_p(entry.ctypes.data), cap)
    if rc < 0:
        raise DetAttnError(rc, "detattn_diag_dkdv_list", last_error())
    if rc == 0:
        return None
    return [[(int(e) >> 1, bool(e & 1)) for e in entry[start[i]:start[i + 1]]] for i in range(nb)]


def diag_exp2(x):
    """(poly, poly pair form, special-function unit) 2^x of a float32 CUDA tensor."""
    _need(x, "x", torch.float32, tuple(x.shape))
    ys = [torch.empty_like(x) for _ in range(3)]
    _check(lib().detattn_diag_exp2(_ptr(x), _ptr(ys[0]), _ptr(ys[1]), _ptr(ys[2]), x.numel(),
                                   _stream()), "detattn_diag_exp2")
    return tuple(ys)


def selftest_wait_timeout(limit_ns: int = 50_000_000):
    """Runs the device-side bounded-wait self-test (see include/detattn.h)."""
    _check(lib().detattn_selftest_wait_timeout(int(limit_ns), _stream()),
           "detattn_selftest_wait_timeout")


def set_dkdv_split(blocks_per_key_tile: int):
    """Forces the dK/dV split (1, 2, 4, 8) or restores automatic (0)."""
    _check(lib().detattn_set_dkdv_split(int(blocks_per_key_tile)), "detattn_set_dkdv_split")


def set_dkdv_deal(mode: int):
    """dK/dV key-tile deal at D = 64: 0 automatic, 1 plain walk, 2 listed deal."""
    _check(lib().detattn_set_dkdv_deal(int(mode)), "detattn_set_dkdv_deal")


def set_wait_limit_ns(ns: int):
    lib().detattn_set_wait_limit_ns(int(ns))
