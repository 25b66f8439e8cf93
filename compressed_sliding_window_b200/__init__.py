"""B200-native Heavily Compressed Attention (HCA) forward path.

Python binding over the C ABI of ``libhca.so`` (declared in include/hca.h).
The functions here only check and marshal arguments (device pointers, sizes,
the current CUDA stream); every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the library is missing or no CUDA
device is present, calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Tuple

import torch

from .build import LIB_PATH

HEADS = 64
HEAD_DIM = 512
BLOCK = 128
WINDOW = 128

STATUS = {
    0: "HCA_OK", 1: "HCA_ERR_INVALID_ARG", 2: "HCA_ERR_UNSUPPORTED", 3: "HCA_ERR_CUDA",
    4: "HCA_ERR_TIMEOUT", 5: "HCA_ERR_DEVICE_INPUT",
}


class HCAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")
        self.code = code


# The C structures of hca.h, native alignment (their pointers are read during the call only)
_PAGED_CACHE = struct.Struct("@6Pqiii4x").pack      # hca_paged_cache_t
_PAGE_TABLE = struct.Struct("@PqiiPPii").pack        # hca_page_table_t
_PAGE_ARRAY = struct.Struct("@Pq").pack              # hca_page_array_t

_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded libhca.so (built in-tree by ``build.py``)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m compressed_sliding_window_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.hca_compress.argtypes = [vp, vp, vp, i, i, vp, vp, vp]
        L.hca_prefill_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, f, vp, vp, vp, sz, vp]
        L.hca_prefill_fwd_vha.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, f, vp, vp, i, vp, vp,
                                          vp, sz, vp]
        L.hca_prefill_workspace_size.argtypes = [i, i]
        L.hca_prefill_workspace_size.restype = sz
        L.hca_decode_workspace_size.argtypes = [i]
        L.hca_decode_workspace_size.restype = sz
        L.hca_decode.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, i, i, f, vp, sz, vp, vp]
        L.hca_prefill_bwd_workspace_size.argtypes = [i, i]
        L.hca_prefill_bwd_workspace_size.restype = sz
        L.hca_prefill_bwd.argtypes = [vp] * 10 + [i, i, i, f] + [vp] * 6 + [sz, vp]
        L.hca_decode_vha.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, i, i, f, vp, vp, i, vp, sz,
                                     vp, vp]
        L.hca_cache_append.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, vp, i, vp]
        L.hca_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, i, i, f, vp, vp, vp, vp, vp, i, vp,
                                      sz, vp, vp]
        L.hca_quantize_e4m3.argtypes = [vp, ctypes.c_longlong, vp, vp, vp]
        L.hca_decode_e4m3.argtypes = [vp, vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, i, i, f, vp,
                                      sz, vp, vp]
        pc = pt = pa = ctypes.c_char_p     # packed structures
        L.hca_paged_append.argtypes = [vp, vp, vp, vp, vp, i, i, pc, vp]
        L.hca_paged_prefill_workspace_size.argtypes = [i, i]
        L.hca_paged_prefill_workspace_size.restype = sz
        L.hca_paged_prefill.argtypes = [vp] * 7 + [i, i, i, f, vp, vp, i, pc, vp, vp, sz, vp]
        L.hca_paged_decode.argtypes = [vp, vp, vp, i, i, f, vp, vp, i, pc, vp, vp, sz, vp]
        L.hca_paged_decode_step.argtypes = [vp] * 6 + [i, i, f, vp, vp, i, pc, vp, vp, sz, vp]
        L.hca_paged_decode_workspace_size.argtypes = [i]
        L.hca_paged_decode_workspace_size.restype = sz
        L.hca_pages_workspace_size.argtypes = [i, i, i]
        L.hca_pages_workspace_size.restype = sz
        L.hca_pages_resize.argtypes = [pt, vp, vp, sz, vp]
        L.hca_pages_resize_copy.argtypes = [pt, vp, pa, i, vp, sz, vp]
        L.hca_pages_fork.argtypes = [pt, vp, vp, vp, i, pa, i, pa, i, vp, vp, sz, vp]
        L.hca_pages_compact.argtypes = [pt, pa, i, vp, vp, sz, vp]
        L.hca_pages_copy.argtypes = [pa, i, i, vp, vp, i, vp, sz, vp]
        L.hca_get_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
        L.hca_selftest_bounded_wait.argtypes = [i, vp]
        L.hca_status_string.argtypes = [i]
        L.hca_status_string.restype = ctypes.c_char_p
        L.hca_version.restype = i
        for name in ("hca_compress", "hca_prefill_fwd", "hca_decode", "hca_get_device_error",
                     "hca_selftest_bounded_wait", "hca_cache_append", "hca_decode_step",
                     "hca_quantize_e4m3", "hca_decode_e4m3", "hca_prefill_fwd_vha",
                     "hca_decode_vha", "hca_prefill_bwd", "hca_paged_append",
                     "hca_paged_prefill", "hca_paged_decode", "hca_paged_decode_step",
                     "hca_pages_resize", "hca_pages_resize_copy", "hca_pages_fork",
                     "hca_pages_compact", "hca_pages_copy"):
            getattr(L, name).restype = i
        _LIB = L
    return _LIB


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _check(t: torch.Tensor, name: str, shape=None, dtype=torch.bfloat16):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _ok(fn: str, code: int):
    if code != 0:
        raise HCAError(fn, code)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def compress(k: torch.Tensor, v: torch.Tensor, s: torch.Tensor,
             ck: Optional[torch.Tensor] = None, cv: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Compressed cache entries for every complete 128-token block.

    k, v: [B, T, 512] bf16; s: [B, T] bf16 -> (ck, cv) [B, T // 128, 512] bf16.
    """
    B, T, D = k.shape
    _check(k, "k", (B, T, HEAD_DIM))
    _check(v, "v", (B, T, HEAD_DIM))
    _check(s, "s", (B, T))
    nb = T // BLOCK
    if ck is None:
        ck = torch.empty((B, nb, HEAD_DIM), dtype=torch.bfloat16, device=k.device)
    if cv is None:
        cv = torch.empty((B, nb, HEAD_DIM), dtype=torch.bfloat16, device=k.device)
    _check(ck, "ck", (B, nb, HEAD_DIM))
    _check(cv, "cv", (B, nb, HEAD_DIM))
    _ok("hca_compress", lib().hca_compress(k.data_ptr(), v.data_ptr(), s.data_ptr(), B, T,
                                           _ptr(ck) if nb else None, _ptr(cv) if nb else None,
                                           _stream(k.device)))
    return ck, cv


def prefill_workspace_size(B: int, T: int) -> int:
    return int(lib().hca_prefill_workspace_size(B, T))


def _check_vha(vha, device):
    down, up = vha
    r = down.shape[1] if down.dim() == 2 else -1
    _check(down, "vha_down", (HEADS, r))
    _check(up, "vha_up", (HEADS, r))
    if not 1 <= r <= HEADS or down.device != device or up.device != device:
        raise ValueError(f"vha factors must be [64, r] bf16 on {device} with 1 <= r <= 64")
    return down, up, r


def prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, ck: torch.Tensor,
            cv: torch.Tensor, g: torch.Tensor, scale: Optional[float] = None,
            out: Optional[torch.Tensor] = None, return_lse: bool = False,
            workspace: Optional[torch.Tensor] = None, vha=None):
    """HCA prefill attention with the gate fused.

    q, g: [B, T, 64, 512]; k, v: [B, T, 512]; ck, cv: [B, T // 128, 512]
    -> out [B, T, 64, 512] bf16 (and lse [B, T, 64] fp32 when asked).
    `vha` = (down, up), each [64, r] bf16: virtual head attention fused into
    the epilogue (hca_prefill_fwd_vha).
    """
    B, T, H, D = q.shape
    _check(q, "q", (B, T, H, HEAD_DIM))
    _check(g, "g", (B, T, H, HEAD_DIM))
    _check(k, "k", (B, T, HEAD_DIM))
    _check(v, "v", (B, T, HEAD_DIM))
    nb = T // BLOCK
    _check(ck, "ck", (B, nb, HEAD_DIM))
    _check(cv, "cv", (B, nb, HEAD_DIM))
    if scale is None:
        scale = 1.0 / math.sqrt(HEAD_DIM)
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", (B, T, H, HEAD_DIM))
    lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        workspace = torch.empty((prefill_workspace_size(B, T),), dtype=torch.uint8,
                                device=q.device)
    _check(workspace, "workspace", dtype=torch.uint8)
    if vha is None:
        _ok("hca_prefill_fwd", lib().hca_prefill_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(ck) if nb else None,
            _ptr(cv) if nb else None, g.data_ptr(), B, T, H, ctypes.c_float(scale),
            out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel(),
            _stream(q.device)))
    else:
        down, up, r = _check_vha(vha, q.device)
        _ok("hca_prefill_fwd_vha", lib().hca_prefill_fwd_vha(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(ck) if nb else None,
            _ptr(cv) if nb else None, g.data_ptr(), B, T, H, ctypes.c_float(scale),
            down.data_ptr(), up.data_ptr(), r, out.data_ptr(), _ptr(lse), workspace.data_ptr(),
            workspace.numel(), _stream(q.device)))
    return (out, lse) if return_lse else out


def prefill_bwd_workspace_size(B: int, T: int) -> int:
    return int(lib().hca_prefill_bwd_workspace_size(B, T))


def prefill_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, s: torch.Tensor,
                     ck: torch.Tensor, cv: torch.Tensor, g: torch.Tensor, out: torch.Tensor,
                     lse: torch.Tensor, dout: torch.Tensor, scale: Optional[float] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Gradients of sum(dout * out) for the HCA prefill (hca_prefill_bwd).

    q, g, out, dout: [B, T, 64, 512] bf16; k, v: [B, T, 512]; s: [B, T];
    ck, cv: the forward's compressed cache; lse: [B, T, 64] fp32 from the
    forward.  Returns dq, dg (bf16, shapes of q and g), dk, dv ([B, T, 512]
    fp32) and ds ([B, T] fp32) as (dq, dk, dv, ds, dg).
    """
    B, T, H, D = q.shape
    for t, n in ((q, "q"), (g, "g"), (out, "out"), (dout, "dout")):
        _check(t, n, (B, T, H, HEAD_DIM))
    _check(k, "k", (B, T, HEAD_DIM))
    _check(v, "v", (B, T, HEAD_DIM))
    _check(s, "s", (B, T))
    nb = T // BLOCK
    _check(ck, "ck", (B, nb, HEAD_DIM))
    _check(cv, "cv", (B, nb, HEAD_DIM))
    _check(lse, "lse", (B, T, H), dtype=torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(HEAD_DIM)
    dq = torch.empty_like(q)
    dg = torch.empty_like(g)
    dk = torch.empty((B, T, HEAD_DIM), dtype=torch.float32, device=q.device)
    dv = torch.empty_like(dk)
    ds = torch.empty((B, T), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty((prefill_bwd_workspace_size(B, T),), dtype=torch.uint8,
                                device=q.device)
    _check(workspace, "workspace", dtype=torch.uint8)
    _ok("hca_prefill_bwd", lib().hca_prefill_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), s.data_ptr(), _ptr(ck) if nb else None,
        _ptr(cv) if nb else None, g.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
        B, T, H, ctypes.c_float(scale), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
        ds.data_ptr(), dg.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _stream(q.device)))
    return dq, dk, dv, ds, dg


def forward(q, k, v, s, g, scale: Optional[float] = None, return_lse: bool = False):
    """Compress then prefill: the whole HCA forward for a prompt."""
    ck, cv = compress(k, v, s)
    return prefill(q, k, v, ck, cv, g, scale=scale, return_lse=return_lse)


def decode_workspace_size(S: int) -> int:
    return int(lib().hca_decode_workspace_size(S))


def decode_workspace(S: int, device) -> torch.Tensor:
    """A zero-filled decode workspace for up to S sequences (reusable across calls)."""
    return torch.zeros((decode_workspace_size(S),), dtype=torch.uint8, device=device)


def decode(q: torch.Tensor, ck: torch.Tensor, cv: torch.Tensor, wk: torch.Tensor,
           wv: torch.Tensor, ctx_len: torch.Tensor, g: torch.Tensor,
           scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, vha=None) -> torch.Tensor:
    """One decode step: q, g [S, 64, 512]; ck, cv [S, max_nc, 512]; wk, wv
    [S, 128, 512] ring windows; ctx_len [S] int32 on the device.  A workspace
    passed in comes from ``decode_workspace`` (zero-filled before first use).
    `vha` = (down, up), each [64, r] bf16: virtual head attention fused into
    the same launch (hca_decode_vha)."""
    S, H, D = q.shape
    _check(q, "q", (S, H, HEAD_DIM))
    _check(g, "g", (S, H, HEAD_DIM))
    max_nc = ck.shape[1]
    _check(ck, "ck", (S, max_nc, HEAD_DIM))
    _check(cv, "cv", (S, max_nc, HEAD_DIM))
    _check(wk, "wk", (S, WINDOW, HEAD_DIM))
    _check(wv, "wv", (S, WINDOW, HEAD_DIM))
    _check(ctx_len, "ctx_len", (S,), dtype=torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(HEAD_DIM)
    if workspace is None:
        workspace = decode_workspace(S, q.device)
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", (S, H, HEAD_DIM))
    _check(workspace, "workspace", dtype=torch.uint8)
    if vha is None:
        _ok("hca_decode", lib().hca_decode(
            q.data_ptr(), _ptr(ck) if max_nc else None, _ptr(cv) if max_nc else None, max_nc,
            wk.data_ptr(), wv.data_ptr(), ctx_len.data_ptr(), g.data_ptr(), S, H,
            ctypes.c_float(scale), workspace.data_ptr(), workspace.numel(), out.data_ptr(),
            _stream(q.device)))
    else:
        down, up, r = _check_vha(vha, q.device)
        _ok("hca_decode_vha", lib().hca_decode_vha(
            q.data_ptr(), _ptr(ck) if max_nc else None, _ptr(cv) if max_nc else None, max_nc,
            wk.data_ptr(), wv.data_ptr(), ctx_len.data_ptr(), g.data_ptr(), S, H,
            ctypes.c_float(scale), down.data_ptr(), up.data_ptr(), r, workspace.data_ptr(),
            workspace.numel(), out.data_ptr(), _stream(q.device)))
    return out


def _check_append(k_new, v_new, s_new, ctx_len, wk, wv, ws, ck, cv):
    S = k_new.shape[0]
    _check(k_new, "k_new", (S, HEAD_DIM))
    _check(v_new, "v_new", (S, HEAD_DIM))
    _check(s_new, "s_new", (S,))
    _check(ctx_len, "ctx_len", (S,), dtype=torch.int32)
    _check(wk, "wk", (S, WINDOW, HEAD_DIM))
    _check(wv, "wv", (S, WINDOW, HEAD_DIM))
    _check(ws, "ws", (S, WINDOW))
    max_nc = ck.shape[1]
    _check(ck, "ck", (S, max_nc, HEAD_DIM))
    _check(cv, "cv", (S, max_nc, HEAD_DIM))
    return S, max_nc


def cache_append(k_new: torch.Tensor, v_new: torch.Tensor, s_new: torch.Tensor,
                 ctx_len: torch.Tensor, wk: torch.Tensor, wv: torch.Tensor, ws: torch.Tensor,
                 ck: torch.Tensor, cv: torch.Tensor) -> None:
    """Append one token per sequence to the decode cache, in place.

    k_new, v_new [S, 512]; s_new [S]; ctx_len [S] int32 (counts the new
    token); wk, wv [S, 128, 512] and ws [S, 128] rings (slot = position mod
    128); ck, cv [S, max_nc, 512]: entry L/128 - 1 is written when L is a
    multiple of 128."""
    S, max_nc = _check_append(k_new, v_new, s_new, ctx_len, wk, wv, ws, ck, cv)
    _ok("hca_cache_append", lib().hca_cache_append(
        k_new.data_ptr(), v_new.data_ptr(), s_new.data_ptr(), ctx_len.data_ptr(), S,
        wk.data_ptr(), wv.data_ptr(), ws.data_ptr(), _ptr(ck) if max_nc else None,
        _ptr(cv) if max_nc else None, max_nc, _stream(k_new.device)))


def decode_step(q: torch.Tensor, g: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                s_new: torch.Tensor, ctx_len: torch.Tensor, wk: torch.Tensor, wv: torch.Tensor,
                ws: torch.Tensor, ck: torch.Tensor, cv: torch.Tensor,
                scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One serving step: cache_append of the new tokens, then decode of their
    queries q, g [S, 64, 512] against the updated cache."""
    S, max_nc = _check_append(k_new, v_new, s_new, ctx_len, wk, wv, ws, ck, cv)
    _check(q, "q", (S, HEADS, HEAD_DIM))
    _check(g, "g", (S, HEADS, HEAD_DIM))
    if scale is None:
        scale = 1.0 / math.sqrt(HEAD_DIM)
    if workspace is None:
        workspace = decode_workspace(S, q.device)
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", (S, HEADS, HEAD_DIM))
    _check(workspace, "workspace", dtype=torch.uint8)
    _ok("hca_decode_step", lib().hca_decode_step(
        q.data_ptr(), g.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), s_new.data_ptr(),
        ctx_len.data_ptr(), S, HEADS, ctypes.c_float(scale), wk.data_ptr(), wv.data_ptr(),
        ws.data_ptr(), _ptr(ck) if max_nc else None, _ptr(cv) if max_nc else None, max_nc,
        workspace.data_ptr(), workspace.numel(), out.data_ptr(), _stream(q.device)))
    return out


def quantize_e4m3(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """FP8 storage of bf16 rows x [..., 512]: (codes uint8 [..., 512], scale
    fp32 [...]), scale = amax / 448 per row, codes = e4m3(x / scale)."""
    if x.shape[-1] != HEAD_DIM:
        raise ValueError(f"x rows must be {HEAD_DIM} wide")
    _check(x, "x", tuple(x.shape))
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rows = x.numel() // HEAD_DIM
    _ok("hca_quantize_e4m3", lib().hca_quantize_e4m3(
        x.data_ptr(), rows, codes.data_ptr(), scale.data_ptr(), _stream(x.device)))
    return codes, scale


def decode_e4m3(q: torch.Tensor, ck: torch.Tensor, ck_scale: torch.Tensor, cv: torch.Tensor,
                cv_scale: torch.Tensor, wk: torch.Tensor, wk_scale: torch.Tensor,
                wv: torch.Tensor, wv_scale: torch.Tensor, ctx_len: torch.Tensor, g: torch.Tensor,
                scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step over an FP8 cache (codes and row scales from
    ``quantize_e4m3``): q, g [S, 64, 512] bf16; ck, cv [S, max_nc, 512] codes
    with [S, max_nc] scales; wk, wv [S, 128, 512] ring codes with [S, 128]
    scales; ctx_len [S] int32."""
    S, H, D = q.shape
    _check(q, "q", (S, H, HEAD_DIM))
    _check(g, "g", (S, H, HEAD_DIM))
    max_nc = ck.shape[1]
    for t, n, shp in ((ck, "ck", (S, max_nc, HEAD_DIM)), (cv, "cv", (S, max_nc, HEAD_DIM)),
                      (wk, "wk", (S, WINDOW, HEAD_DIM)), (wv, "wv", (S, WINDOW, HEAD_DIM))):
        _check(t, n, shp, dtype=torch.uint8)
    for t, n, shp in ((ck_scale, "ck_scale", (S, max_nc)), (cv_scale, "cv_scale", (S, max_nc)),
                      (wk_scale, "wk_scale", (S, WINDOW)), (wv_scale, "wv_scale", (S, WINDOW))):
        _check(t, n, shp, dtype=torch.float32)
    _check(ctx_len, "ctx_len", (S,), dtype=torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(HEAD_DIM)
    if workspace is None:
        workspace = decode_workspace(S, q.device)
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", (S, H, HEAD_DIM))
    _check(workspace, "workspace", dtype=torch.uint8)
    _ok("hca_decode_e4m3", lib().hca_decode_e4m3(
        q.data_ptr(), _ptr(ck) if max_nc else None, _ptr(ck_scale) if max_nc else None,
        _ptr(cv) if max_nc else None, _ptr(cv_scale) if max_nc else None, max_nc,
        wk.data_ptr(), wk_scale.data_ptr(), wv.data_ptr(), wv_scale.data_ptr(),
        ctx_len.data_ptr(), g.data_ptr(), S, H, ctypes.c_float(scale), workspace.data_ptr(),
        workspace.numel(), out.data_ptr(), _stream(q.device)))
    return out


# ---------------------------------------------------------------------------
# Paged cache
# ---------------------------------------------------------------------------
# Every function here first hands its arguments to the compiled module (built with the
# library from csrc/paged_calls.cpp), which checks them and makes the call in one go: 8 of
# the 20 us that a serving step takes on the host when the checks below run one by one.
# False means that it did not make the call (arguments that are not exactly as the
# library takes them, or an option it leaves to this code): the checks below then say
# what is wrong, or make the call themselves.
PAGE_SIZES = (16, 32, 64, 128)
_SCALE = 1.0 / math.sqrt(HEAD_DIM)


_CALLS = None


def _calls():
    """The compiled module (linked against libhca.so, which must be built, and torch)."""
    global _CALLS
    if _CALLS is None:
        lib()
        rebuild = ("build it for torch " + torch.__version__ + " with "
                   "`python -m compressed_sliding_window_b200.build`")
        try:
            from . import _paged_calls
        except ImportError as e:
            raise RuntimeError(f"_paged_calls cannot be loaded ({e}): {rebuild}") from e
        built = getattr(_paged_calls, "torch_version", "another version")
        if built != str(torch.__version__):
            raise RuntimeError(f"_paged_calls was built for torch {built}: {rebuild}")
        _CALLS = _paged_calls
    return _CALLS


def _raise(name: str, code: int):
    raise HCAError(name, code)


def _need(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """_check, and that t lies on `device`, at the cost of a few attribute reads: a
    serving step checks a dozen tensors while the GPU waits for its launch.  Returns
    the data pointer."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        return t.data_ptr()
    _check(t, name, shape, dtype=dtype)
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _device_of(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.device


def _rows(t: torch.Tensor, name: str, dims: int) -> int:
    """Rows of a tensor that has `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimension(s), got shape {tuple(t.shape)}")
    return t.shape[0]


def _call(device: torch.device, name: str, *args):
    """A library call on the current stream of `device`, made the current device for it."""
    if torch.cuda.current_device() == device.index:
        code = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            code = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if code != 0:
        raise HCAError(name, code)


def _sized(device: torch.device, name: str, *args) -> int:
    """A workspace size, which depends on the device."""
    if torch.cuda.current_device() == device.index:
        return int(getattr(lib(), name)(*args))
    with torch.cuda.device(device):
        return int(getattr(lib(), name)(*args))


def _cuda(device) -> torch.device:
    device = torch.device(device)
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


def _workspace(workspace: torch.Tensor, device):
    n = _rows(workspace, "workspace", 1)
    return _need(workspace, "workspace", (n,), torch.uint8, device), n


def _check_table(page_table: torch.Tensor, rows: int, device):
    """A page table: int32 [rows, max_pages] whose rows may lie apart (a view)."""
    if (not isinstance(page_table, torch.Tensor) or page_table.dtype is not torch.int32
            or page_table.dim() != 2 or page_table.shape[0] != rows):
        raise ValueError(f"page_table must be an int32 tensor [{rows}, max_pages]")
    if page_table.device != device:
        raise ValueError(f"page_table is on {page_table.device}, expected {device}")
    cols = page_table.shape[1]
    stride = page_table.stride(0) if rows > 1 else cols
    if (cols > 1 and page_table.stride(1) != 1) or stride < cols:
        raise ValueError("page_table's rows must be contiguous and not overlap")
    return cols, stride


def _paged_cache(S, wk, wv, ws, ck_pages, cv_pages, page_table, device) -> bytes:
    bf16 = torch.bfloat16
    ring = (S, WINDOW, HEAD_DIM)
    pk = _need(wk, "wk", ring, bf16, device)
    pv = _need(wv, "wv", ring, bf16, device)
    ps = 0 if ws is None else _need(ws, "ws", (S, WINDOW), bf16, device)
    if not isinstance(ck_pages, torch.Tensor) or ck_pages.dim() != 3:
        raise ValueError("ck_pages must be [num_pages, page_size, 512]")
    num, size, _ = ck_pages.shape
    if size not in PAGE_SIZES:
        raise ValueError(f"pages must hold 16, 32, 64 or 128 entries, got {size}")
    pool = (num, size, HEAD_DIM)
    pck = _need(ck_pages, "ck_pages", pool, bf16, device)
    pcv = _need(cv_pages, "cv_pages", pool, bf16, device)
    cols, stride = _check_table(page_table, S, device)
    return _PAGED_CACHE(pk, pv, ps, pck if num else 0, pcv if num else 0,
                        page_table.data_ptr() if cols else 0, stride, cols, num, size)


def _check_chunk(k_new, v_new, s_new, q_start, ctx_len, device):
    """(pointers of k_new, v_new, s_new, q_start, ctx_len, then S, N)"""
    S = _rows(ctx_len, "ctx_len", 1)
    N = _rows(k_new, "k_new", 2)
    bf16 = torch.bfloat16
    pl = _need(ctx_len, "ctx_len", (S,), torch.int32, device)
    pk = _need(k_new, "k_new", (N, HEAD_DIM), bf16, device)
    pv = _need(v_new, "v_new", (N, HEAD_DIM), bf16, device)
    ps = _need(s_new, "s_new", (N,), bf16, device)
    pq = None
    if q_start is not None:
        pq = _need(q_start, "q_start", (S + 1,), torch.int32, device)
    elif N != S:
        raise ValueError(f"{N} new tokens for {S} sequences need q_start")
    return pk, pv, ps, pq, pl, S, N


def _attend_args(q, g, out, vha, rows, scale, device):
    """(pointers of q and g, out, its pointer, scale, head-mix factors and rank)"""
    shape = (rows, HEADS, HEAD_DIM)
    pq = _need(q, "q", shape, torch.bfloat16, device)
    pg = _need(g, "g", shape, torch.bfloat16, device)
    if out is None:
        out = torch.empty_like(q)
        po = out.data_ptr()
    else:
        po = _need(out, "out", shape, torch.bfloat16, device)
    down, up, r = (None, None, 0) if vha is None else _check_vha(vha, device)
    return pq, pg, out, po, _SCALE if scale is None else scale, _ptr(down), _ptr(up), r


def paged_append(k_new: torch.Tensor, v_new: torch.Tensor, s_new: torch.Tensor,
                 q_start: Optional[torch.Tensor], ctx_len: torch.Tensor, wk: torch.Tensor,
                 wv: torch.Tensor, ws: torch.Tensor, ck_pages: torch.Tensor,
                 cv_pages: torch.Tensor, page_table: torch.Tensor) -> None:
    """Append a chunk of new tokens per sequence to a paged cache, in place.

    k_new, v_new [N, 512]; s_new [N]: the tokens of all sequences, packed;
    sequence i brings q_start[i] .. q_start[i + 1] - 1 (q_start [S + 1] int32;
    None: one token each).  ctx_len [S] int32 counts them.  wk, wv
    [S, 128, 512] and ws [S, 128] rings; ck_pages, cv_pages
    [num_pages, page_size, 512]; page_table [S, max_pages] int32: entry j of
    sequence i is row j % page_size of page page_table[i, j // page_size]."""
    r = _calls().paged_append(k_new, v_new, s_new, q_start, ctx_len, wk, wv, ws, ck_pages, cv_pages,
                              page_table)
    if r is not False:
        return None if r is None else _raise("hca_paged_append", r)
    device = _device_of(wk, "wk")
    chunk = _check_chunk(k_new, v_new, s_new, q_start, ctx_len, device)
    S, N = chunk[5:]
    cache = _paged_cache(S, wk, wv, ws, ck_pages, cv_pages, page_table, device)
    if N > 0:
        _call(device, "hca_paged_append", *chunk, cache)


def paged_prefill_workspace(S: int, N: int, device) -> torch.Tensor:
    """A zero-filled workspace for paged_prefill of up to N new tokens of up to S sequences
    (reusable across calls)."""
    device = _cuda(device)
    return torch.zeros((_sized(device, "hca_paged_prefill_workspace_size", S, N),),
                       dtype=torch.uint8, device=device)


def paged_prefill(q: torch.Tensor, g: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                  s_new: torch.Tensor, q_start: torch.Tensor, ctx_len: torch.Tensor,
                  wk: torch.Tensor, wv: torch.Tensor, ws: torch.Tensor, ck_pages: torch.Tensor,
                  cv_pages: torch.Tensor, page_table: torch.Tensor, scale: Optional[float] = None,
                  workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  vha=None) -> torch.Tensor:
    """paged_append of a chunk, and the attention of its tokens over the cache.

    q, g [N, 64, 512], packed like k_new -> out [N, 64, 512] bf16 (memory of
    its own; rows before q_start[0] and from q_start[S] on are not written).
    The other arguments are paged_append's;
    `workspace` comes from paged_prefill_workspace; `vha` as for decode."""
    if vha is None and workspace is not None:
        r = _calls().paged_prefill(q, g, k_new, v_new, s_new, q_start, ctx_len, wk, wv, ws, ck_pages,
                                   cv_pages, page_table, scale, workspace, out)
        if r is not False:
            return r if type(r) is not int else _raise("hca_paged_prefill", r)
    device = _device_of(wk, "wk")
    if q_start is None:
        raise ValueError("paged_prefill needs q_start (paged_decode_step takes one token each)")
    chunk = _check_chunk(k_new, v_new, s_new, q_start, ctx_len, device)
    S, N = chunk[5:]
    cache = _paged_cache(S, wk, wv, ws, ck_pages, cv_pages, page_table, device)
    pq, pg, out, po, scale, down, up, r = _attend_args(q, g, out, vha, N, scale, device)
    if N == 0:
        return out
    if workspace is None:
        workspace = paged_prefill_workspace(S, N, device)
    _call(device, "hca_paged_prefill", pq, pg, *chunk, HEADS, scale, down, up, r, cache, po,
          *_workspace(workspace, device))
    return out


def paged_decode_workspace(S: int, device) -> torch.Tensor:
    """A zero-filled workspace for paged_decode of up to S sequences (reusable across calls)."""
    device = _cuda(device)
    return torch.zeros((_sized(device, "hca_paged_decode_workspace_size", S),),
                       dtype=torch.uint8, device=device)


def paged_decode(q: torch.Tensor, ck_pages: torch.Tensor, cv_pages: torch.Tensor,
                 page_table: torch.Tensor, wk: torch.Tensor, wv: torch.Tensor,
                 ctx_len: torch.Tensor, g: torch.Tensor, scale: Optional[float] = None,
                 workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 vha=None) -> torch.Tensor:
    """decode over a paged cache: one query per sequence, q, g [S, 64, 512];
    the cache (see paged_append) already holds its token.  A workspace passed
    in comes from paged_decode_workspace."""
    if vha is None and workspace is not None:
        r = _calls().paged_decode(q, ck_pages, cv_pages, page_table, wk, wv, ctx_len, g, scale,
                                  workspace, out)
        if r is not False:
            return r if type(r) is not int else _raise("hca_paged_decode", r)
    device = _device_of(wk, "wk")
    S = _rows(ctx_len, "ctx_len", 1)
    pl = _need(ctx_len, "ctx_len", (S,), torch.int32, device)
    cache = _paged_cache(S, wk, wv, None, ck_pages, cv_pages, page_table, device)
    pq, pg, out, po, scale, down, up, r = _attend_args(q, g, out, vha, S, scale, device)
    if workspace is None:
        workspace = paged_decode_workspace(S, device)
    _call(device, "hca_paged_decode", pq, pg, pl, S, HEADS, scale, down, up, r, cache, po,
          *_workspace(workspace, device))
    return out


def paged_decode_step(q: torch.Tensor, g: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                      s_new: torch.Tensor, ctx_len: torch.Tensor, wk: torch.Tensor,
                      wv: torch.Tensor, ws: torch.Tensor, ck_pages: torch.Tensor,
                      cv_pages: torch.Tensor, page_table: torch.Tensor,
                      scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, vha=None) -> torch.Tensor:
    """One serving step: paged_append of one token per sequence (k_new, v_new
    [S, 512]; s_new [S]), then paged_decode of their queries q, g [S, 64, 512]."""
    if vha is None and workspace is not None:
        r = _calls().paged_decode_step(q, g, k_new, v_new, s_new, ctx_len, wk, wv, ws, ck_pages,
                                       cv_pages, page_table, scale, workspace, out)
        if r is not False:
            return r if type(r) is not int else _raise("hca_paged_decode_step", r)
    device = _device_of(wk, "wk")
    pk, pv, ps, _, pl, S, _ = _check_chunk(k_new, v_new, s_new, None, ctx_len, device)
    cache = _paged_cache(S, wk, wv, ws, ck_pages, cv_pages, page_table, device)
    pq, pg, out, po, scale, down, up, r = _attend_args(q, g, out, vha, S, scale, device)
    if workspace is None:
        workspace = paged_decode_workspace(S, device)
    _call(device, "hca_paged_decode_step", pq, pg, pk, pv, ps, pl, S, HEADS, scale, down, up, r,
          cache, po, *_workspace(workspace, device))
    return out


def _page_table(page_table, n_pages, ref, page_size: int, device):
    """(the packed hca_page_table_t, rows, pages)"""
    if page_size not in PAGE_SIZES:
        raise ValueError(f"pages must hold 16, 32, 64 or 128 entries, got {page_size}")
    rows, num = _rows(n_pages, "n_pages", 1), _rows(ref, "ref", 1)
    pn = _need(n_pages, "n_pages", (rows,), torch.int32, device)
    pr = _need(ref, "ref", (num,), torch.int32, device)
    cols, stride = _check_table(page_table, rows, device)
    return (_PAGE_TABLE(page_table.data_ptr(), stride, rows, cols, pn, pr, num, page_size), rows,
            num)


def _page_arrays(arrays, items: int, what: str, device) -> bytes:
    """Item arrays for the library: any dtype, contiguous, [items, ...]."""
    out = b""
    for i, t in enumerate(arrays):
        if not isinstance(t, torch.Tensor) or t.device != device:
            raise ValueError(f"{what}[{i}] must be a tensor on {device}")
        if not t.is_contiguous() or t.dim() < 2 or t.shape[0] != items:
            raise ValueError(f"{what}[{i}] must be contiguous [{items}, ...], got {tuple(t.shape)}")
        nbytes = t.nbytes // items
        if nbytes < 16 or nbytes % 16:
            raise ValueError(f"{what}[{i}]: items of {nbytes} bytes, a multiple of 16 is needed")
        out += _PAGE_ARRAY(t.data_ptr(), nbytes)
    return out


def _pages_workspace(workspace, rows, num_pages, n, device):
    if workspace is None:
        size = lib().hca_pages_workspace_size(rows, num_pages, n)
        workspace = torch.empty((size,), dtype=torch.uint8, device=device)
    return workspace


def resize_pages(page_table: torch.Tensor, n_pages: torch.Tensor, ref: torch.Tensor,
                 entries: torch.Tensor, page_size: int,
                 workspace: Optional[torch.Tensor] = None, pools=()) -> None:
    """Give every row of the page table the pages of entries[r] entries, in place.

    page_table [R, max_pages], n_pages [R], ref [num_pages], entries [R], all
    int32 on the device.  0 frees a row, a negative number leaves it.  Rows
    shrink first; rows that grow take the lowest free pages, row by row, while
    there are any (n_pages[r] tells what row r has).

    A row that is cut inside a page it shares with a branch may only be
    appended to with a page of its own: pass the `pools` ([num_pages, ...]
    tensors), and its partly used page is replaced by a copy in each of them.
    (Without them the row keeps the shared page, which then must not be
    written.)  Where no page is free for that, device_error() reports it and
    the row keeps the shared page."""
    if not len(pools):
        r = _calls().resize_pages(page_table, n_pages, ref, entries, page_size, workspace)
        if r is not False:
            return None if r is None else _raise("hca_pages_resize", r)
    device = _device_of(page_table, "page_table")
    table, rows, num = _page_table(page_table, n_pages, ref, page_size, device)
    pe = _need(entries, "entries", (rows,), torch.int32, device)
    workspace = _pages_workspace(workspace, rows, num, 0, device)
    if len(pools):
        _call(device, "hca_pages_resize_copy", table, pe, _page_arrays(pools, num, "pools", device),
              len(pools), *_workspace(workspace, device))
    else:
        _call(device, "hca_pages_resize", table, pe, *_workspace(workspace, device))


def fork_pages(page_table: torch.Tensor, n_pages: torch.Tensor, ref: torch.Tensor,
               parents: torch.Tensor, children: torch.Tensor, entries: torch.Tensor, pools,
               page_size: int, rings=(), workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Branch sequences: the empty row children[i] becomes a copy of parents[i]
    at entries[i] entries (parents, children, entries [n] int32).

    Full pages are shared; the partly filled one is copied in every pool
    ([num_pages, ...] tensors), and row parents[i] of every ring ([R, ...]) to
    row children[i].  Returns ok [n] int32: 0 where no page was free (or the
    pair was refused, which device_error() reports)."""
    r = _calls().fork_pages(page_table, n_pages, ref, parents, children, entries, pools, page_size,
                            rings, workspace)
    if r is not False:
        return r if type(r) is not int else _raise("hca_pages_fork", r)
    device = _device_of(page_table, "page_table")
    table, rows, num = _page_table(page_table, n_pages, ref, page_size, device)
    n = _rows(parents, "parents", 1)
    pp = _need(parents, "parents", (n,), torch.int32, device)
    pc = _need(children, "children", (n,), torch.int32, device)
    pe = _need(entries, "entries", (n,), torch.int32, device)
    pool_arrays = _page_arrays(pools, num, "pools", device)
    ring_arrays = _page_arrays(rings, rows, "rings", device)
    ok = torch.empty((n,), dtype=torch.int32, device=device)
    if n == 0:
        return ok
    workspace = _pages_workspace(workspace, rows, num, n, device)
    _call(device, "hca_pages_fork", table, pp, pc, pe, n, pool_arrays, len(pools), ring_arrays,
          len(rings), ok.data_ptr(), *_workspace(workspace, device))
    return ok


def compact_pages(page_table: torch.Tensor, n_pages: torch.Tensor, ref: torch.Tensor, pools,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Close up a pool: the pages in use take the lowest numbers, page_table,
    ref and the contents of every pool ([num_pages, ...]) follow.  Returns the
    number of pages in use ([1] int32 on the device); all others are free."""
    r = _calls().compact_pages(page_table, n_pages, ref, pools, PAGE_SIZES[0], workspace)
    if r is not False:
        return r if type(r) is not int else _raise("hca_pages_compact", r)
    device = _device_of(page_table, "page_table")
    table, rows, num = _page_table(page_table, n_pages, ref, PAGE_SIZES[0], device)
    arrays = _page_arrays(pools, num, "pools", device)
    live = torch.empty((1,), dtype=torch.int32, device=device)
    workspace = _pages_workspace(workspace, rows, num, 0, device)
    _call(device, "hca_pages_compact", table, arrays, len(pools), live.data_ptr(),
          *_workspace(workspace, device))
    return live


def copy_pages(arrays, src: torch.Tensor, dst: torch.Tensor,
               workspace: Optional[torch.Tensor] = None) -> None:
    """Copy item src[i] to item dst[i] of every array ([items, ...] tensors of
    any dtype; src, dst [n] int32).  Pairs out of range, and all pairs whose
    destination is named twice or is also a source, are left out and reported
    by device_error()."""
    if len(arrays) == 0:
        return
    device = _device_of(arrays[0], "arrays[0]")
    n, items = _rows(src, "src", 1), arrays[0].shape[0] if arrays[0].dim() else 0
    ps = _need(src, "src", (n,), torch.int32, device)
    pd = _need(dst, "dst", (n,), torch.int32, device)
    item_arrays = _page_arrays(arrays, items, "arrays", device)
    if n == 0:
        return
    workspace = _pages_workspace(workspace, 1, items, n, device)
    _call(device, "hca_pages_copy", item_arrays, len(arrays), items, ps, pd, n,
          *_workspace(workspace, device))


def device_error(device: Optional[torch.device] = None) -> Tuple[int, int]:
    """(status, where) from the device-side error word (synchronises the stream)."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    where = ctypes.c_uint(0)
    code = lib().hca_get_device_error(_stream(device), ctypes.byref(where))
    return code, where.value


def selftest_bounded_wait(limit_us: int, device: Optional[torch.device] = None):
    device = device or torch.device("cuda", torch.cuda.current_device())
    _ok("hca_selftest_bounded_wait", lib().hca_selftest_bounded_wait(limit_us, _stream(device)))
