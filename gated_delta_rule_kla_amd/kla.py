"""Thin ctypes binding over libkla.so (include/kla.h).

Argument marshalling only: shape/dtype checks, output allocation with torch
and the current HIP stream.  Every step of the operator runs in the HIP
kernels; there is no fallback.  If libkla.so is missing the call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

__all__ = ["chunk_fwd", "chunk_workspace_bytes", "chunk_fwd_workspace_bytes", "pgdn_chunk_fwd", "pgdn_decode_step",
           "pgdn_chunk_workspace_bytes",
           "GAINS", "decode_step", "gdn_chunk_fwd", "gdn_decode_step", "chunk_bwd",
           "gdn_chunk_bwd", "chunk_bwd_workspace_bytes", "glr_chunk_fwd", "glr_chunk_bwd", "glr_decode_step",
           "glr_chunk_workspace_bytes", "la_chunk_fwd", "la_chunk_bwd", "la_decode_step",
           "la_chunk_workspace_bytes", "attn_fwd", "kv4_append", "kv4_read", "kv4_cache", "attn_kv4_decode_step",
           "attn_kv4_decode_workspace_bytes", "attn_kv4_chunk_fwd", "attn_kv4_chunk_workspace_bytes",
           "attn_kv4_weigh", "kv4_weights", "kv4_evict", "kv4_evict_workspace_bytes", "lib", "lib_path", "KlaError", "KLA_DT_BF16",
           "KLA_DT_F32"]

KLA_DT_BF16 = 0
KLA_DT_F32 = 1
GAINS = {"given": 0, "kaczmarz": 1}  # kla_gain_t
_DTYPES = {torch.bfloat16: KLA_DT_BF16, torch.float32: KLA_DT_F32}

_LIB: Optional[ctypes.CDLL] = None


def lib_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkla.so")


class KlaError(RuntimeError):
    """A negative kla_status_t returned by the library."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libkla.so once.  torch is imported first so that the library binds
    to the HIP runtime torch already mapped (same soname)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is not built: run `python -c 'import __graft_entry__ as g; g.build()'` "
                "(or python gated_delta_rule_kla_amd/build.py)")
        L = ctypes.CDLL(path)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.kla_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp,
                                    i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.kla_chunk_fwd.restype = i32
        L.kla_chunk_workspace_bytes.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, i32]
        L.kla_chunk_workspace_bytes.restype = sz
        L.kla_chunk_fwd_seg.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp,
                                        i32, i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.kla_chunk_fwd_seg.restype = i32
        L.kla_chunk_seg_workspace_bytes.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32]
        L.kla_chunk_seg_workspace_bytes.restype = sz
        L.kla_decode_step.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp,
                                      i32, i32, i32, i32, i32, vp]
        L.kla_decode_step.restype = i32
        L.kla_gdn_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.kla_gdn_chunk_fwd.restype = i32
        L.kla_gdn_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        L.kla_gdn_decode_step.restype = i32
        L.kla_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                    i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.kla_chunk_bwd.restype = i32
        L.kla_gdn_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.kla_gdn_chunk_bwd.restype = i32
        L.kla_chunk_bwd_workspace_bytes.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, i32]
        L.kla_chunk_bwd_workspace_bytes.restype = sz
        L.kla_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp,
                                            i32, i32, i32, i32, i32, i32, i32, i32, vp]
        L.kla_chunk_fwd_noalloc.restype = i32
        L.kla_chunk_fwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        L.kla_chunk_fwd_workspace_bytes.restype = sz
        L.kla_pgdn_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, f32, i32, f32, vp, vp, vp, vp, vp, vp, vp,
                                         i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.kla_pgdn_chunk_fwd.restype = i32
        L.kla_pgdn_chunk_workspace_bytes.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, i32]
        L.kla_pgdn_chunk_workspace_bytes.restype = sz
        L.kla_pgdn_decode_step.argtypes = [vp, vp, vp, vp, vp, f32, i32, f32, vp, vp, vp,
                                           i32, i32, i32, i32, i32, vp]
        L.kla_pgdn_decode_step.restype = i32
        L.kla_glr_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.kla_glr_chunk_fwd.restype = i32
        L.kla_glr_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, sz,
                                        vp]
        L.kla_glr_chunk_bwd.restype = i32
        L.kla_glr_chunk_workspace_bytes.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32]
        L.kla_glr_chunk_workspace_bytes.restype = sz
        L.kla_glr_decode_step.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.kla_glr_decode_step.restype = i32
        L.kla_la_chunk_fwd.argtypes = [vp] * 10 + [i32] * 7 + [vp, sz, vp]
        L.kla_la_chunk_fwd.restype = i32
        L.kla_la_chunk_bwd.argtypes = [vp] * 15 + [i32] * 7 + [vp, sz, vp]
        L.kla_la_chunk_bwd.restype = i32
        for f in (L.kla_la_chunk_workspace_bytes, L.kla_la_chunk_bwd_workspace_bytes):
            f.argtypes = [vp, vp] + [i32] * 7
            f.restype = sz
        L.kla_la_decode_step.argtypes = [vp] * 7 + [i32] * 5 + [vp]
        L.kla_la_decode_step.restype = i32
        L.kla_attn_fwd.argtypes = [vp, vp, vp, f32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, vp]
        L.kla_attn_fwd.restype = i32
        for f in (L.kla_kv4_append, L.kla_kv4_read):
            f.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32, vp]
            f.restype = i32
        L.kla_attn_kv4_decode_step.argtypes = [vp, vp, vp, vp, vp, f32, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                               i32, vp, sz, vp]
        L.kla_attn_kv4_decode_step.restype = i32
        L.kla_attn_kv4_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        L.kla_attn_kv4_decode_workspace_bytes.restype = sz
        L.kla_attn_kv4_chunk_fwd.argtypes = [vp] * 5 + [f32] + [vp] * 4 + [i32] * 11 + [vp, sz, vp]
        L.kla_attn_kv4_chunk_fwd.restype = i32
        L.kla_attn_kv4_chunk_workspace_bytes.argtypes = [vp, vp] + [i32] * 8
        L.kla_attn_kv4_chunk_workspace_bytes.restype = sz
        L.kla_attn_kv4_weigh.argtypes = [vp] * 6 + [f32] + [vp] * 3 + [i32] * 12 + [vp]
        L.kla_attn_kv4_weigh.restype = i32
        L.kla_kv4_evict.argtypes = [vp] * 7 + [i32] * 9 + [vp, sz, vp]
        L.kla_kv4_evict.restype = i32
        L.kla_kv4_evict_workspace_bytes.argtypes = [i32] * 6
        L.kla_kv4_evict_workspace_bytes.restype = sz
        L.kla_status_str.argtypes = [i32]
        L.kla_status_str.restype = ctypes.c_char_p
        L.kla_abi_version.argtypes = []
        L.kla_abi_version.restype = i32
        _LIB = L
    return _LIB


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise KlaError(fn, status, lib().kla_status_str(status).decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _chunk_call(fn: str, q, k, v, g, coef, eps, initial_state, cu_seqlens, chunk, output_final_state,
                cu_seqlens_host, out, final_state, workspace, seg_chunks=None):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"kla.{fn} needs GPU tensors")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    _need(q, "q", dtype, (B, H, T, dk), dev)
    _need(k, "k", dtype, (B, H, T, dk), dev)
    _need(v, "v", dtype, (B, H, T, dv), dev)
    _need(g, "g", dtype, (B, H, T), dev)
    _need(coef, "eta" if eps is not None else "beta", dtype, (B, H, T), dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        if cu_seqlens_host is None:
            cu_seqlens_host = cu_seqlens.cpu()
        cu_seqlens_host = cu_seqlens_host.to(torch.int32).contiguous()
        if cu_seqlens_host.numel() != cu_seqlens.numel():
            raise ValueError("cu_seqlens_host does not mirror cu_seqlens")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, H, dk, dv), dev)
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=dtype, device=dev)
    else:
        _need(out, "out", dtype, (B, H, T, dv), dev)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (N, H, dk, dv), dev)
    host_ptr = None if cu_seqlens_host is None else cu_seqlens_host.data_ptr()
    if isinstance(workspace, str) and workspace == "static" and eps is not None:
        # kla_chunk_fwd_noalloc: the library's fixed per-GPU scratch, no workspace argument
        st = lib().kla_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), float(eps),
                                         _ptr(initial_state), _ptr(out), _ptr(final_state), _ptr(cu_seqlens),
                                         host_ptr, N, B, H, T, dk, dv, int(chunk), _DTYPES[dtype], _stream(dev))
        _check("kla_chunk_fwd_noalloc", st)
        return out, final_state
    if isinstance(workspace, str):
        raise ValueError(f"kla.{fn}: workspace must be a tensor or None ('static' is for chunk_fwd only)")
    if seg_chunks is not None:
        if eps is None:
            raise ValueError(f"kla.{fn}: seg_chunks is for chunk_fwd only")
        ws_bytes = lib().kla_chunk_seg_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, int(chunk),
                                                       _DTYPES[dtype], int(seg_chunks))
    else:
        ws_bytes = lib().kla_chunk_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, int(chunk),
                                                   _DTYPES[dtype])
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    tail = (_ptr(initial_state), _ptr(out), _ptr(final_state), _ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv,
            int(chunk), _DTYPES[dtype], _ptr(workspace), workspace.numel(), _stream(dev))
    if seg_chunks is not None:
        st = lib().kla_chunk_fwd_seg(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), float(eps), *tail[:13],
                                     int(seg_chunks), *tail[13:])
        _check("kla_chunk_fwd_seg", st)
    elif eps is not None:
        st = lib().kla_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), float(eps), *tail)
        _check("kla_chunk_fwd", st)
    else:
        st = lib().kla_gdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), *tail)
        _check("kla_gdn_chunk_fwd", st)
    return out, final_state


def chunk_fwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    eta: torch.Tensor,
    eps: float = 1e-6,
    initial_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    chunk: int = 64,
    output_final_state: bool = True,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    out: Optional[torch.Tensor] = None,
    final_state: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
    seg_chunks: Optional[int] = None,
) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """KLA chunkwise prefill (kla_chunk_fwd).

    q, k: [B, H, T, dk]; v: [B, H, T, dv]; g, eta: [B, H, T]; all bf16 or all
    fp32 on one GPU.  initial_state: [N, H, dk, dv] fp32 or None.  cu_seqlens:
    int32 [N + 1] on the GPU (B must be 1) or None.  Returns (o, final_state).
    ``final_state`` may be passed as the same tensor as ``initial_state`` to
    update it in place.  ``workspace`` (uint8, on the GPU, at least
    chunk_workspace_bytes(...) bytes) is taken from torch's caching allocator
    on the current stream when not given.  ``workspace="static"`` calls
    kla_chunk_fwd_noalloc instead, which uses the library's fixed per-GPU
    scratch buffer (KLA_NOALLOC_SCRATCH_BYTES, 64 MiB) and allocates nothing
    (pass ``out`` and ``final_state`` to keep the call allocation-free here too).
    ``seg_chunks`` (kla_chunk_fwd_seg): None lets the library choose whether to cut
    long sequences into segments scanned side by side; 0 never cuts; n > 0 cuts
    every sequence into segments of n chunks.
    """
    if seg_chunks is not None and isinstance(workspace, str):
        raise ValueError("kla.chunk_fwd: seg_chunks needs a workspace tensor or None")
    return _chunk_call("chunk_fwd", q, k, v, g, eta, eps, initial_state, cu_seqlens, chunk,
                       output_final_state, cu_seqlens_host, out, final_state, workspace, seg_chunks)


NOALLOC_SCRATCH_BYTES = 64 << 20  # KLA_NOALLOC_SCRATCH_BYTES in include/kla.h


def gdn_chunk_fwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    beta: torch.Tensor,
    initial_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    chunk: int = 64,
    output_final_state: bool = True,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    out: Optional[torch.Tensor] = None,
    final_state: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated delta rule chunkwise prefill (kla_gdn_chunk_fwd): as chunk_fwd
    with the update coefficient ``beta`` [B, H, T] given instead of eta, eps."""
    return _chunk_call("gdn_chunk_fwd", q, k, v, g, beta, None, initial_state, cu_seqlens, chunk,
                       output_final_state, cu_seqlens_host, out, final_state, workspace)


def chunk_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int, chunk: int = 64,
                          dtype: torch.dtype = torch.bfloat16,
                          cu_seqlens_host: Optional[torch.Tensor] = None,
                          seg_chunks: Optional[int] = None) -> int:
    """Workspace bytes kla_chunk_fwd needs (kla_chunk_workspace_bytes), or
    kla_chunk_fwd_seg with ``seg_chunks`` (kla_chunk_seg_workspace_bytes); 0 for
    arguments it would reject.  With packed sequences pass the host int32
    cu_seqlens (B must be 1)."""
    if cu_seqlens_host is not None:
        cu = cu_seqlens_host.to(torch.int32).contiguous()
        # the device pointer is only tested for NULL here
        args = (ctypes.c_void_p(16), cu.data_ptr(), cu.numel() - 1, B, H, T, dk, dv, int(chunk), _DTYPES[dtype])
    else:
        args = (None, None, B, B, H, T, dk, dv, int(chunk), _DTYPES[dtype])
    if seg_chunks is not None:
        return lib().kla_chunk_seg_workspace_bytes(*args, int(seg_chunks))
    return lib().kla_chunk_workspace_bytes(*args)


def pgdn_chunk_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int, chunk: int = 64,
                               dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes kla_pgdn_chunk_fwd needs for a dense batch
    (kla_pgdn_chunk_workspace_bytes); 0 where it runs the general kernel."""
    return lib().kla_pgdn_chunk_workspace_bytes(None, None, B, B, H, T, dk, dv, int(chunk), _DTYPES[dtype])


def chunk_fwd_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int, chunk: int = 64,
                              num_seqs: Optional[int] = None) -> int:
    """Upper bound on the workspace bytes kla_chunk_fwd needs for these sizes,
    for either dtype and either layout (kla_chunk_fwd_workspace_bytes)."""
    return lib().kla_chunk_fwd_workspace_bytes(B, H, T, dk, dv, int(chunk), B if num_seqs is None else num_seqs)


def _bwd_call(fn, q, k, v, g, coef, eps, do, initial_state, dfinal_state, cu_seqlens, chunk, cu_seqlens_host,
              need_dinitial, workspace):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"kla.{fn} needs GPU tensors")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    _need(q, "q", dtype, (B, H, T, dk), dev)
    _need(k, "k", dtype, (B, H, T, dk), dev)
    _need(v, "v", dtype, (B, H, T, dv), dev)
    _need(g, "g", dtype, (B, H, T), dev)
    _need(coef, "eta" if eps is not None else "beta", dtype, (B, H, T), dev)
    _need(do, "do", dtype, (B, H, T, dv), dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        if cu_seqlens_host is None:
            cu_seqlens_host = cu_seqlens.cpu()
        cu_seqlens_host = cu_seqlens_host.to(torch.int32).contiguous()
        if cu_seqlens_host.numel() != cu_seqlens.numel():
            raise ValueError("cu_seqlens_host does not mirror cu_seqlens")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, H, dk, dv), dev)
    if dfinal_state is not None:
        _need(dfinal_state, "dfinal_state", torch.float32, (N, H, dk, dv), dev)
    dq = torch.empty_like(q)
    dkk = torch.empty_like(k)
    dvv = torch.empty_like(v)
    dg = torch.empty((B, H, T), dtype=torch.float32, device=dev)
    dcoef = torch.empty((B, H, T), dtype=torch.float32, device=dev)
    ds0 = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if need_dinitial else None
    host_ptr = None if cu_seqlens_host is None else cu_seqlens_host.data_ptr()
    ws_bytes = lib().kla_chunk_bwd_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, int(chunk),
                                                   _DTYPES[dtype])
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    mid = (_ptr(initial_state), _ptr(do), _ptr(dfinal_state), _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dg),
           _ptr(dcoef), _ptr(ds0), _ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, int(chunk),
           _DTYPES[dtype], _ptr(workspace), workspace.numel(), _stream(dev))
    if eps is not None:
        st = lib().kla_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), float(eps), *mid)
        _check("kla_chunk_bwd", st)
    else:
        st = lib().kla_gdn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), *mid)
        _check("kla_gdn_chunk_bwd", st)
    return dq, dkk, dvv, dg, dcoef, ds0


def chunk_bwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    eta: torch.Tensor,
    do: torch.Tensor,
    eps: float = 1e-6,
    initial_state: Optional[torch.Tensor] = None,
    dfinal_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    chunk: int = 64,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    need_dinitial: bool = True,
    workspace: Optional[torch.Tensor] = None,
):
    """Gradients of chunk_fwd (kla_chunk_bwd) for upstream gradients ``do``
    [B, H, T, dv] (dtype of q) and ``dfinal_state`` [N, H, dk, dv] fp32 or None.

    Returns (dq, dk, dv, dg, deta, dinitial_state): dq, dk, dv in the inputs'
    dtype; dg, deta [B, H, T] fp32; dinitial_state [N, H, dk, dv] fp32 (None
    unless ``need_dinitial``).  Other arguments as chunk_fwd.
    """
    return _bwd_call("chunk_bwd", q, k, v, g, eta, eps, do, initial_state, dfinal_state, cu_seqlens, chunk,
                     cu_seqlens_host, need_dinitial, workspace)


def gdn_chunk_bwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    beta: torch.Tensor,
    do: torch.Tensor,
    initial_state: Optional[torch.Tensor] = None,
    dfinal_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    chunk: int = 64,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    need_dinitial: bool = True,
    workspace: Optional[torch.Tensor] = None,
):
    """Gradients of gdn_chunk_fwd (kla_gdn_chunk_bwd); the fifth result is dbeta."""
    return _bwd_call("gdn_chunk_bwd", q, k, v, g, beta, None, do, initial_state, dfinal_state, cu_seqlens,
                     chunk, cu_seqlens_host, need_dinitial, workspace)


def chunk_bwd_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int, chunk: int = 64,
                              dtype: torch.dtype = torch.bfloat16,
                              cu_seqlens_host: Optional[torch.Tensor] = None) -> int:
    """Workspace bytes kla_chunk_bwd needs (kla_chunk_bwd_workspace_bytes)."""
    if cu_seqlens_host is not None:
        cu = cu_seqlens_host.to(torch.int32).contiguous()
        return lib().kla_chunk_bwd_workspace_bytes(ctypes.c_void_p(16), cu.data_ptr(), cu.numel() - 1, B, H, T,
                                                   dk, dv, int(chunk), _DTYPES[dtype])
    return lib().kla_chunk_bwd_workspace_bytes(None, None, B, B, H, T, dk, dv, int(chunk), _DTYPES[dtype])


def _decode_call(fn, q, k, v, g, coef, eps, state, out):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"kla.{fn} needs GPU tensors")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    N, H, dk = q.shape
    dv = v.shape[-1]
    _need(q, "q", dtype, (N, H, dk), dev)
    _need(k, "k", dtype, (N, H, dk), dev)
    _need(v, "v", dtype, (N, H, dv), dev)
    _need(g, "g", dtype, (N, H), dev)
    _need(coef, "eta" if eps is not None else "beta", dtype, (N, H), dev)
    _need(state, "state", torch.float32, (N, H, dk, dv), dev)
    if out is None:
        out = torch.empty((N, H, dv), dtype=dtype, device=dev)
    else:
        _need(out, "out", dtype, (N, H, dv), dev)
    tail = (_ptr(state), _ptr(out), N, H, dk, dv, _DTYPES[dtype], _stream(dev))
    if eps is not None:
        st = lib().kla_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), float(eps), *tail)
        _check("kla_decode_step", st)
    else:
        st = lib().kla_gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), *tail)
        _check("kla_gdn_decode_step", st)
    return out


def decode_step(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    eta: torch.Tensor,
    eps: float,
    state: torch.Tensor,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """One KLA recurrent step (kla_decode_step); ``state`` is updated in place.

    q, k: [N, H, dk]; v: [N, H, dv]; g, eta: [N, H]; state: [N, H, dk, dv] fp32.
    Returns o [N, H, dv].
    """
    return _decode_call("decode_step", q, k, v, g, eta, eps, state, out)


def gdn_decode_step(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    beta: torch.Tensor,
    state: torch.Tensor,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """One gated-delta-rule step (kla_gdn_decode_step): as decode_step with the
    update coefficient ``beta`` [N, H] given; ``state`` is updated in place."""
    return _decode_call("gdn_decode_step", q, k, v, g, beta, None, state, out)


def pgdn_chunk_fwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    coef: torch.Tensor,
    eps: float = 1e-6,
    gain: str = "given",
    band: float = 1.5,
    initial_state: Optional[torch.Tensor] = None,
    initial_acc: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    chunk: int = 64,
    output_final_state: bool = True,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    out: Optional[torch.Tensor] = None,
    final_state: Optional[torch.Tensor] = None,
    final_acc: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
):
    """Preconditioned gated delta rule prefill (kla_pgdn_chunk_fwd).

    As chunk_fwd, with ``coef`` [B, H, T] the update coefficient beta
    (gain="given") or eta (gain="kaczmarz": beta = eta / (k . w + eps)), the
    preconditioner's band x >= 1, and the key accumulator [N, H, dk] fp32 in
    (``initial_acc``, zeros when None) and out.  ``workspace`` (uint8, at least
    kla_pgdn_chunk_workspace_bytes(...) bytes) is taken from torch's caching
    allocator when not given.  Returns (o, final_state, final_acc) (the last two
    None unless ``output_final_state`` or given)."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("kla.pgdn_chunk_fwd needs GPU tensors")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if gain not in GAINS:
        raise ValueError(f"gain must be one of {sorted(GAINS)}")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    for t, name, shp in ((q, "q", (B, H, T, dk)), (k, "k", (B, H, T, dk)), (v, "v", (B, H, T, dv)),
                         (g, "g", (B, H, T)), (coef, "coef", (B, H, T))):
        _need(t, name, dtype, shp, dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        if cu_seqlens_host is None:
            cu_seqlens_host = cu_seqlens.cpu()
        cu_seqlens_host = cu_seqlens_host.to(torch.int32).contiguous()
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, H, dk, dv), dev)
    if initial_acc is not None:
        _need(initial_acc, "initial_acc", torch.float32, (N, H, dk), dev)
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=dtype, device=dev)
    _need(out, "out", dtype, (B, H, T, dv), dev)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if output_final_state and final_acc is None:
        final_acc = torch.empty((N, H, dk), dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (N, H, dk, dv), dev)
    if final_acc is not None:
        _need(final_acc, "final_acc", torch.float32, (N, H, dk), dev)
    host_ptr = None if cu_seqlens_host is None else cu_seqlens_host.data_ptr()
    ws_bytes = lib().kla_pgdn_chunk_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, int(chunk),
                                                    _DTYPES[dtype])
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    st = lib().kla_pgdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), float(eps), GAINS[gain],
                                  float(band), _ptr(initial_state), _ptr(initial_acc), _ptr(out), _ptr(final_state),
                                  _ptr(final_acc), _ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, int(chunk),
                                  _DTYPES[dtype], _ptr(workspace), workspace.numel(), _stream(dev))
    _check("kla_pgdn_chunk_fwd", st)
    return out, final_state, final_acc


def pgdn_decode_step(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    coef: torch.Tensor,
    eps: float,
    state: torch.Tensor,
    acc: torch.Tensor,
    gain: str = "given",
    band: float = 1.5,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """One preconditioned gated-delta-rule step (kla_pgdn_decode_step);
    ``state`` [N, H, dk, dv] and ``acc`` [N, H, dk] (fp32) are updated in place."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("kla.pgdn_decode_step needs GPU tensors")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if gain not in GAINS:
        raise ValueError(f"gain must be one of {sorted(GAINS)}")
    N, H, dk = q.shape
    dv = v.shape[-1]
    for t, name, shp in ((q, "q", (N, H, dk)), (k, "k", (N, H, dk)), (v, "v", (N, H, dv)), (g, "g", (N, H)),
                         (coef, "coef", (N, H))):
        _need(t, name, dtype, shp, dev)
    _need(state, "state", torch.float32, (N, H, dk, dv), dev)
    _need(acc, "acc", torch.float32, (N, H, dk), dev)
    if out is None:
        out = torch.empty((N, H, dv), dtype=dtype, device=dev)
    _need(out, "out", dtype, (N, H, dv), dev)
    st = lib().kla_pgdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(coef), float(eps), GAINS[gain],
                                    float(band), _ptr(state), _ptr(acc), _ptr(out), N, H, dk, dv, _DTYPES[dtype],
                                    _stream(dev))
    _check("kla_pgdn_decode_step", st)
    return out


def _fit(t, name: str, dtype, shape, dev) -> None:
    """_need's check, in the order that costs least where everything is fine."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _need(t, name, dtype, shape, dev)


def _device_of(fn: str, t: torch.Tensor) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"kla.{fn}: expected a tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"kla.{fn} needs GPU tensors")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return t.device


_INT32 = 0x7FFFFFFF  # sizes go to the library as 32-bit integers


def _rank(t: torch.Tensor, name: str, rank: int) -> tuple:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != rank:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {rank} dimensions")
    if max(t.shape) > _INT32:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: a dimension of more than {_INT32}")
    return tuple(t.shape)


def _seqlens(cu_seqlens, cu_seqlens_host, B: int, dev):
    """Number of sequences and the host mirror of cu_seqlens (None for a dense batch)."""
    if cu_seqlens is None:
        if cu_seqlens_host is not None:
            raise ValueError("cu_seqlens_host without cu_seqlens")
        return B, None
    n = cu_seqlens.numel()
    _fit(cu_seqlens, "cu_seqlens", torch.int32, (n,), dev)
    if n == 0:
        raise ValueError("cu_seqlens must hold at least one offset")
    host = cu_seqlens if cu_seqlens_host is None else cu_seqlens_host
    if host.numel() != n:
        raise ValueError("cu_seqlens_host does not mirror cu_seqlens")
    if host.is_cuda or host.dtype is not torch.int32 or not host.is_contiguous():
        host = host.to("cpu", torch.int32).contiguous()
    return n - 1, host


def _optional(t, name, dtype, shape, dev) -> None:
    if t is not None:
        _fit(t, name, dtype, shape, dev)


def _scratch(workspace, need: int, dev) -> Optional[torch.Tensor]:
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev or workspace.dtype != torch.uint8 \
            or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace


def _call(fn: str, dev: torch.device, *args) -> None:
    """Call the library on the current stream of the tensors' device, which need not be the
    current device."""
    f, index = getattr(lib(), fn), dev.index
    if index == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        _check(fn, st)


def glr_chunk_workspace_bytes(B: int, H: int, T: int, d: int, dtype: torch.dtype = torch.bfloat16,
                              cu_seqlens_host: Optional[torch.Tensor] = None) -> int:
    """Workspace bytes glr_chunk_fwd and glr_chunk_bwd need (kla_glr_chunk_workspace_bytes)."""
    if cu_seqlens_host is not None:
        cu = cu_seqlens_host.to("cpu", torch.int32).contiguous()
        # the device pointer is only tested for NULL here
        return lib().kla_glr_chunk_workspace_bytes(ctypes.c_void_p(16), cu.data_ptr(), cu.numel() - 1, B, H, T, d,
                                                   _DTYPES[dtype])
    return lib().kla_glr_chunk_workspace_bytes(None, None, B, B, H, T, d, _DTYPES[dtype])


def glr_chunk_fwd(
    x: torch.Tensor,
    g: torch.Tensor,
    initial_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    output_final_state: bool = True,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    out: Optional[torch.Tensor] = None,
    final_state: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated linear recurrence over whole sequences (kla_glr_chunk_fwd): per channel
    h_t = exp(g_t) h_{t-1} + x_t, o_t = h_t.

    x, g: [B, H, T, d], bf16 or fp32; initial_state: [N, H, d] fp32 or None; cu_seqlens: int32
    [N + 1] on the GPU (B must be 1) or None, with its host mirror to avoid a copy back.
    The mirror sizes the call, the offsets on the GPU decide: a captured call may be replayed with
    others.  Returns (o, final_state); ``final_state`` may be passed as the same tensor as
    ``initial_state``.
    """
    dev = _device_of("glr_chunk_fwd", x)
    dtype = x.dtype
    B, H, T, d = shape = _rank(x, "x", 4)
    _fit(x, "x", dtype, shape, dev)
    _fit(g, "g", dtype, shape, dev)
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, B, dev)
    _optional(initial_state, "initial_state", torch.float32, (N, H, d), dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _fit(out, "out", dtype, shape, dev)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, H, d), dtype=torch.float32, device=dev)
    _optional(final_state, "final_state", torch.float32, (N, H, d), dev)
    host_ptr = _ptr(host)
    ws = _scratch(workspace, lib().kla_glr_chunk_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, d,
                                                                 _DTYPES[dtype]), dev)
    _call("kla_glr_chunk_fwd", dev, _ptr(x), _ptr(g), _ptr(initial_state), _ptr(out), _ptr(final_state),
          _ptr(cu_seqlens), host_ptr, N, B, H, T, d, _DTYPES[dtype], _ptr(ws), 0 if ws is None else ws.numel())
    return out, final_state


def glr_chunk_bwd(
    g: torch.Tensor,
    o: torch.Tensor,
    do: torch.Tensor,
    initial_state: Optional[torch.Tensor] = None,
    dfinal_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    need_dinitial: bool = True,
    workspace: Optional[torch.Tensor] = None,
):
    """Gradients of glr_chunk_fwd (kla_glr_chunk_bwd) from its output ``o`` and the upstream
    gradients ``do`` [B, H, T, d] and ``dfinal_state`` [N, H, d] fp32 or None.

    Returns (dx, dg, dinitial_state): dx, dg in the inputs' dtype, dinitial_state [N, H, d]
    fp32 (None unless ``need_dinitial``).
    """
    dev = _device_of("glr_chunk_bwd", g)
    dtype = g.dtype
    B, H, T, d = shape = _rank(g, "g", 4)
    for t, name in ((g, "g"), (o, "o"), (do, "do")):
        _fit(t, name, dtype, shape, dev)
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, B, dev)
    _optional(initial_state, "initial_state", torch.float32, (N, H, d), dev)
    _optional(dfinal_state, "dfinal_state", torch.float32, (N, H, d), dev)
    dx, dg = torch.empty_like(g), torch.empty_like(g)
    dh0 = torch.empty((N, H, d), dtype=torch.float32, device=dev) if need_dinitial else None
    host_ptr = _ptr(host)
    ws = _scratch(workspace, lib().kla_glr_chunk_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, d,
                                                                 _DTYPES[dtype]), dev)
    _call("kla_glr_chunk_bwd", dev, _ptr(g), _ptr(o), _ptr(initial_state), _ptr(do), _ptr(dfinal_state), _ptr(dx),
          _ptr(dg), _ptr(dh0), _ptr(cu_seqlens), host_ptr, N, B, H, T, d, _DTYPES[dtype], _ptr(ws),
          0 if ws is None else ws.numel())
    return dx, dg, dh0


def glr_decode_step(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the gated linear recurrence (kla_glr_decode_step): x, g [N, H, d];
    ``state`` [N, H, d] fp32 is updated in place.  Returns o [N, H, d]."""
    if not (isinstance(x, torch.Tensor) and isinstance(g, torch.Tensor) and isinstance(state, torch.Tensor)
            and x.is_cuda and x.dtype in _DTYPES and g.dtype is x.dtype and state.dtype is torch.float32
            and x.dim() == 3 and x.shape == g.shape == state.shape and x.device == g.device == state.device
            and x.is_contiguous() and g.is_contiguous() and state.is_contiguous()):
        _refuse_glr_step(x, g, state)
    dev, (N, H, d) = x.device, x.shape
    if N > _INT32 or H > _INT32 or d > _INT32:
        _refuse_glr_step(x, g, state)
    if out is None:
        out = torch.empty_like(x)
    else:
        _fit(out, "out", x.dtype, x.shape, dev)
    _call("kla_glr_decode_step", dev, x.data_ptr(), g.data_ptr(), state.data_ptr(), out.data_ptr(), N, H, d,
          _DTYPES[x.dtype])
    return out


# The single-token calls check their tensors in one expression, since their host time counts;
# where it fails, these name what is wrong.
def _refuse_glr_step(x, g, state) -> None:
    dev = _device_of("glr_decode_step", x)
    shape = _rank(x, "x", 3)
    _need(x, "x", x.dtype, shape, dev)
    _need(g, "g", x.dtype, shape, dev)
    _need(state, "state", torch.float32, shape, dev)


def _decays(g, dtype, shape, dev):
    """Pointers of g [*shape] in the inputs' dtype, or of per-head log-decays [H] in fp32."""
    if isinstance(g, torch.Tensor) and g.dim() == 1:
        _fit(g, "g", torch.float32, (shape[1],), dev)
        return None, g.data_ptr()
    _fit(g, "g", dtype, shape, dev)
    return g.data_ptr(), None


def la_chunk_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int, dtype: torch.dtype = torch.bfloat16,
                             cu_seqlens_host: Optional[torch.Tensor] = None, backward: bool = False) -> int:
    """Workspace bytes la_chunk_fwd, or la_chunk_bwd, needs (kla_la_chunk_workspace_bytes)."""
    f = lib().kla_la_chunk_bwd_workspace_bytes if backward else lib().kla_la_chunk_workspace_bytes
    if cu_seqlens_host is not None:
        cu = cu_seqlens_host.to("cpu", torch.int32).contiguous()
        # the device pointer is only tested for NULL here
        return f(ctypes.c_void_p(16), cu.data_ptr(), cu.numel() - 1, B, H, T, dk, dv, _DTYPES[dtype])
    return f(None, None, B, B, H, T, dk, dv, _DTYPES[dtype])


def la_chunk_fwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    initial_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    output_final_state: bool = True,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    out: Optional[torch.Tensor] = None,
    final_state: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay per head over whole sequences (kla_la_chunk_fwd):
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.

    q, k: [B, H, T, dk]; v: [B, H, T, dv], bf16 or fp32; g: [B, H, T] in their dtype, or [H] fp32
    for decays that are the same for all tokens of a head; initial_state: [N, H, dk, dv] fp32 or
    None; cu_seqlens: int32 [N + 1] on the GPU (B must be 1) or None, with its host mirror to avoid
    a copy back.  The mirror sizes the call, the offsets on the GPU decide: a captured call may be
    replayed with others.  Returns (o, final_state); ``final_state`` may be passed as the same
    tensor as ``initial_state``.
    """
    dev = _device_of("la_chunk_fwd", q)
    dtype = q.dtype
    B, H, T, dk = shape = _rank(q, "q", 4)
    dv = _rank(v, "v", 4)[3]
    _fit(q, "q", dtype, shape, dev)
    _fit(k, "k", dtype, shape, dev)
    _fit(v, "v", dtype, (B, H, T, dv), dev)
    each, fixed = _decays(g, dtype, (B, H, T), dev)
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, B, dev)
    _optional(initial_state, "initial_state", torch.float32, (N, H, dk, dv), dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _fit(out, "out", dtype, (B, H, T, dv), dev)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    _optional(final_state, "final_state", torch.float32, (N, H, dk, dv), dev)
    host_ptr, dt = _ptr(host), _DTYPES[dtype]
    ws = _scratch(workspace, lib().kla_la_chunk_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, dt), dev)
    _call("kla_la_chunk_fwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), each, fixed, _ptr(initial_state),
          out.data_ptr(), _ptr(final_state), _ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, dt, _ptr(ws),
          0 if ws is None else ws.numel())
    return out, final_state


def la_chunk_bwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    do: torch.Tensor,
    initial_state: Optional[torch.Tensor] = None,
    dfinal_state: Optional[torch.Tensor] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    need_dinitial: bool = True,
    workspace: Optional[torch.Tensor] = None,
):
    """Gradients of la_chunk_fwd (kla_la_chunk_bwd) from its inputs and the upstream gradients
    ``do`` [B, H, T, dv] and ``dfinal_state`` [N, H, dk, dv] fp32 or None.

    Returns (dq, dk, dv, dg, dinitial_state): the first four shaped and typed as q, k, v and g
    ([H] fp32 log-decays have the sum over all tokens), dinitial_state fp32 (None unless
    ``need_dinitial``).
    """
    dev = _device_of("la_chunk_bwd", q)
    dtype = q.dtype
    B, H, T, dk = shape = _rank(q, "q", 4)
    dv = _rank(v, "v", 4)[3]
    _fit(q, "q", dtype, shape, dev)
    _fit(k, "k", dtype, shape, dev)
    _fit(v, "v", dtype, (B, H, T, dv), dev)
    _fit(do, "do", dtype, (B, H, T, dv), dev)
    each, fixed = _decays(g, dtype, (B, H, T), dev)
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, B, dev)
    _optional(initial_state, "initial_state", torch.float32, (N, H, dk, dv), dev)
    _optional(dfinal_state, "dfinal_state", torch.float32, (N, H, dk, dv), dev)
    dq, dk_, dv_, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g)
    ds0 = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if need_dinitial else None
    host_ptr, dt = _ptr(host), _DTYPES[dtype]
    ws = _scratch(workspace, lib().kla_la_chunk_bwd_workspace_bytes(_ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, dt),
                  dev)
    _call("kla_la_chunk_bwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), each, fixed, _ptr(initial_state),
          do.data_ptr(), _ptr(dfinal_state), dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(), dg.data_ptr(), _ptr(ds0),
          _ptr(cu_seqlens), host_ptr, N, B, H, T, dk, dv, dt, _ptr(ws), 0 if ws is None else ws.numel())
    return dq, dk_, dv_, dg, ds0


def la_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of linear attention (kla_la_decode_step): q, k [N, H, dk], v [N, H, dv], g [N, H]
    in their dtype or [H] fp32; ``state`` [N, H, dk, dv] fp32 is updated in place.  Returns
    o [N, H, dv]."""
    if not (isinstance(q, torch.Tensor) and isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor)
            and isinstance(g, torch.Tensor) and isinstance(state, torch.Tensor) and q.is_cuda and q.dtype in _DTYPES
            and k.dtype is v.dtype is q.dtype and state.dtype is torch.float32 and q.dim() == 3 and v.dim() == 3
            and q.shape == k.shape and state.shape == q.shape + v.shape[2:] and v.shape[:2] == q.shape[:2]
            and q.device == k.device == v.device == g.device == state.device and q.is_contiguous()
            and k.is_contiguous() and v.is_contiguous() and state.is_contiguous()):
        _refuse_la_step(q, k, v, state)
    dev, (N, H, dk), dv = q.device, q.shape, v.shape[2]
    if N > _INT32 or H > _INT32 or dk > _INT32 or dv > _INT32:
        _refuse_la_step(q, k, v, state)
    each, fixed = _decays(g, q.dtype, (N, H), dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _fit(out, "out", q.dtype, v.shape, dev)
    _call("kla_la_decode_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), each, fixed, state.data_ptr(),
          out.data_ptr(), N, H, dk, dv, _DTYPES[q.dtype])
    return out


def _refuse_la_step(q, k, v, state) -> None:
    dev = _device_of("la_decode_step", q)
    N, H, dk = _rank(q, "q", 3)
    dv = _rank(v, "v", 3)[2]
    _need(q, "q", q.dtype, (N, H, dk), dev)
    _need(k, "k", q.dtype, (N, H, dk), dev)
    _need(v, "v", q.dtype, (N, H, dv), dev)
    _need(state, "state", torch.float32, (N, H, dk, dv), dev)


def attn_fwd(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    scale: Optional[float] = None,
    cu_seqlens: Optional[torch.Tensor] = None,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    cu_seqlens_k: Optional[torch.Tensor] = None,
    cu_seqlens_k_host: Optional[torch.Tensor] = None,
    out: Optional[torch.Tensor] = None,
    lse: Optional[torch.Tensor] = None,
) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal softmax attention over whole prompts (kla_attn_fwd).

    q: [B, Hq, Tq, D]; k, v: [B, Hkv, Tk, D], bf16 or fp32, Hq a multiple of Hkv; scale:
    D ** -0.5 when None.  cu_seqlens: int32 [N + 1] packs the queries of N sequences (B must be
    1), cu_seqlens_k their keys (None: the same offsets); the last query of a sequence sees its
    last key.  Returns (o, lse): lse [B, Hq, Tq] fp32, the logarithm of each query's sum.
    """
    dev = _device_of("attn_fwd", q)
    dtype = q.dtype
    B, Hq, Tq, D = shape = _rank(q, "q", 4)
    _, Hkv, Tk, _ = _rank(k, "k", 4)
    _fit(q, "q", dtype, shape, dev)
    _fit(k, "k", dtype, (B, Hkv, Tk, D), dev)
    _fit(v, "v", dtype, (B, Hkv, Tk, D), dev)
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, B, dev)
    if cu_seqlens_k is None:
        if cu_seqlens_k_host is not None:
            raise ValueError("cu_seqlens_k_host without cu_seqlens_k")
        host_k = None
    else:
        Nk, host_k = _seqlens(cu_seqlens_k, cu_seqlens_k_host, B, dev)
        if cu_seqlens is None or Nk != N:
            raise ValueError("cu_seqlens_k needs cu_seqlens of as many sequences")
    if out is None:
        out = torch.empty_like(q)
    else:
        _fit(out, "out", dtype, shape, dev)
    if lse is None:
        lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=dev)
    else:
        _fit(lse, "lse", torch.float32, (B, Hq, Tq), dev)
    _call("kla_attn_fwd", dev, _ptr(q), _ptr(k), _ptr(v), D ** -0.5 if scale is None else float(scale), _ptr(out),
          _ptr(lse), _ptr(cu_seqlens), _ptr(host), _ptr(cu_seqlens_k), _ptr(host_k), N, B, Hq, Hkv, Tq, Tk, D,
          _DTYPES[dtype])
    return out, lse


def kv4_cache(num_pages: int, Hkv: int, page_size: int, D: int, device) -> Tuple[torch.Tensor, torch.Tensor]:
    """An empty 4-bit key/value cache: (codes [num_pages, 2, Hkv, page_size, D/2], scales
    [num_pages, 2, Hkv, page_size, D/32]), uint8 (the format: kla_kv4_append in include/kla.h)."""
    return (torch.zeros(num_pages, 2, Hkv, page_size, D // 2, dtype=torch.uint8, device=device),
            torch.zeros(num_pages, 2, Hkv, page_size, D // 32, dtype=torch.uint8, device=device))


def _cache_args(codes, scales, block_table, N: int, dev):
    """Sizes of a cache and its block table: (num_pages, Hkv, page_size, D, max_pages)."""
    if (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and isinstance(block_table, torch.Tensor)
            and codes.dim() == 5 and block_table.dim() == 2):
        P, two, H, page, half = codes.shape
        M = block_table.shape[1]
        if (two == 2 and scales.shape == (P, 2, H, page, half // 16) and block_table.shape[0] == N
                and codes.dtype is scales.dtype is torch.uint8 and block_table.dtype is torch.int32
                and codes.device == scales.device == block_table.device == dev
                and codes.is_contiguous() and scales.is_contiguous() and block_table.is_contiguous()):
            return P, H, page, 2 * half, M
    P, two, Hkv, page, half = _rank(codes, "codes", 5)
    if two != 2:
        raise ValueError(f"codes has shape {tuple(codes.shape)}, expected [num_pages, 2, Hkv, page_size, D/2]")
    _need(codes, "codes", torch.uint8, (P, 2, Hkv, page, half), dev)
    _need(scales, "scales", torch.uint8, (P, 2, Hkv, page, half // 16), dev)
    _, M = _rank(block_table, "block_table", 2)
    _need(block_table, "block_table", torch.int32, (N, M), dev)
    return P, Hkv, page, 2 * half, M


def kv4_append(
    k: torch.Tensor,
    v: torch.Tensor,
    codes: torch.Tensor,
    scales: torch.Tensor,
    block_table: torch.Tensor,
    start: torch.Tensor,
    cu_seqlens: Optional[torch.Tensor] = None,
    cu_seqlens_host: Optional[torch.Tensor] = None,
) -> None:
    """Store keys and values in a 4-bit cache (kla_kv4_append), in place.

    k, v: [B, Hkv, T, D], bf16 or fp32; codes, scales: as kv4_cache makes them; block_table:
    int32 [N, max_pages]; start: int32 [N], the tokens that each sequence holds already (negative:
    the sequence is padding); cu_seqlens as in chunk_fwd (None: N = B).  Rows behind the last
    sequence of the offsets on the GPU are not stored.
    """
    if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and k.is_cuda and k.dtype in _DTYPES
            and v.dtype is k.dtype and k.dim() == 4 and v.shape == k.shape and v.device == k.device
            and k.is_contiguous() and v.is_contiguous()):
        _need(k, "k", k.dtype, _rank(k, "k", 4), _device_of("kv4_append", k))
        _need(v, "v", k.dtype, k.shape, k.device)
    dev, (B, Hkv, T, D) = k.device, k.shape
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, B, dev)
    P, H, page, Dc, M = _cache_args(codes, scales, block_table, N, dev)
    if (H, Dc) != (Hkv, D):
        raise ValueError(f"k has {Hkv} heads of {D} channels, the cache {H} of {Dc}")
    _fit(start, "start", torch.int32, (N,), dev)
    _call("kla_kv4_append", dev, k.data_ptr(), v.data_ptr(), codes.data_ptr(), scales.data_ptr(),
          block_table.data_ptr(), start.data_ptr(), _ptr(cu_seqlens), _ptr(host), N, B, Hkv, T, D, P, page, M, _DTYPES[k.dtype])


def kv4_read(
    codes: torch.Tensor,
    scales: torch.Tensor,
    block_table: torch.Tensor,
    start: torch.Tensor,
    cu_seqlens: torch.Tensor,
    dtype: torch.dtype = torch.bfloat16,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
) -> Tuple[torch.Tensor, torch.Tensor]:
    """The values that a 4-bit cache holds (kla_kv4_read): k, v [1, Hkv, T, D] of positions
    start[n] ... start[n] + length of sequence n, packed by cu_seqlens (int32 [N + 1], T its
    last; its host mirror avoids a copy back).  ``out``: (k, v) to write to, whose rows behind the
    last sequence of the offsets on the GPU stay as they are."""
    if not isinstance(codes, torch.Tensor) or codes.device.type != "cuda":
        raise ValueError("kla.kv4_read needs GPU tensors")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    dev = codes.device
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, 1, dev)
    if host is None:
        raise ValueError("kla.kv4_read needs cu_seqlens")
    P, Hkv, page, D, M = _cache_args(codes, scales, block_table, N, dev)
    _fit(start, "start", torch.int32, (N,), dev)
    T = ctypes.c_int32.from_address(host.data_ptr() + 4 * N).value  # host[-1]
    shape = (1, Hkv, max(T, 0), D)
    if out is None:
        k = torch.empty(shape, dtype=dtype, device=dev)
        out = (k, torch.empty_like(k))
    else:
        _fit(out[0], "out[0]", dtype, shape, dev)
        _fit(out[1], "out[1]", dtype, shape, dev)
    _call("kla_kv4_read", dev, out[0].data_ptr(), out[1].data_ptr(), codes.data_ptr(), scales.data_ptr(),
          block_table.data_ptr(), start.data_ptr(), cu_seqlens.data_ptr(), host.data_ptr(), N, 1, Hkv, T, D, P, page, M, _DTYPES[dtype])
    return out


_MAX_LEN = _INT32 - 65536  # the longest max_len


def attn_kv4_decode_workspace_bytes(N: int, Hq: int, Hkv: int, D: int, max_len: int,
                                    dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes attn_kv4_decode_step needs (kla_attn_kv4_decode_workspace_bytes)."""
    return lib().kla_attn_kv4_decode_workspace_bytes(N, Hq, Hkv, D, min(int(max_len), _INT32), _DTYPES[dtype])


def attn_kv4_decode_step(
    q: torch.Tensor,
    codes: torch.Tensor,
    scales: torch.Tensor,
    block_table: torch.Tensor,
    seq_lens: torch.Tensor,
    scale: Optional[float] = None,
    max_len: Optional[int] = None,
    out: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """Attention of one token per sequence over a 4-bit cache (kla_attn_kv4_decode_step).

    q: [N, Hq, D], bf16 or fp32; seq_lens: int32 [N] cached tokens, the new one's among them;
    scale: D ** -0.5 when None; max_len: a bound on seq_lens known to the host (the block
    table's room when None; a tight one makes fewer, fuller workgroups).  Returns o [N, Hq, D].
    """
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dtype in _DTYPES and q.dim() == 3 and q.is_contiguous()):
        _need(q, "q", q.dtype, _rank(q, "q", 3), _device_of("attn_kv4_decode_step", q))
    dev, shape = q.device, q.shape
    N, Hq, D = shape
    P, Hkv, page, Dc, M = _cache_args(codes, scales, block_table, N, dev)
    if Dc != D:
        raise ValueError(f"q has {D} channels, the cache {Dc}")
    _fit(seq_lens, "seq_lens", torch.int32, (N,), dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _fit(out, "out", q.dtype, shape, dev)
    max_len = min(M * page, _MAX_LEN) if max_len is None else min(int(max_len), _INT32)
    dt = _DTYPES[q.dtype]
    ws = _scratch(workspace, lib().kla_attn_kv4_decode_workspace_bytes(N, Hq, Hkv, D, max_len, dt), dev)
    _call("kla_attn_kv4_decode_step", dev, q.data_ptr(), codes.data_ptr(), scales.data_ptr(), block_table.data_ptr(),
          seq_lens.data_ptr(), D ** -0.5 if scale is None else float(scale), out.data_ptr(), N, Hq, Hkv, D, P, page, M, max_len, dt, _ptr(ws),
          0 if ws is None else ws.numel())
    return out


def _chunk_args(fn: str, q, codes, scales, block_table, seq_lens, cu_seqlens, cu_seqlens_host, max_len):
    """Checked sizes of a call of new tokens over the cache."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dtype in _DTYPES and q.dim() == 4 and q.is_contiguous()):
        _need(q, "q", q.dtype, _rank(q, "q", 4), _device_of(fn, q))
    dev, (B, Hq, T, D) = q.device, q.shape
    if max(q.shape) > _INT32:
        _rank(q, "q", 4)
    N, host = _seqlens(cu_seqlens, cu_seqlens_host, B, dev)
    P, Hkv, page, Dc, M = _cache_args(codes, scales, block_table, N, dev)
    if Dc != D:
        raise ValueError(f"q has {D} channels, the cache {Dc}")
    _fit(seq_lens, "seq_lens", torch.int32, (N,), dev)
    max_len = min(M * page, _MAX_LEN) if max_len is None else min(int(max_len), _INT32)
    return dev, N, host, (N, B, Hq, Hkv, T, D), (P, page, M, max_len)


def attn_kv4_chunk_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, D: int, max_len: int,
                                   dtype: torch.dtype = torch.bfloat16,
                                   cu_seqlens_host: Optional[torch.Tensor] = None) -> int:
    """Workspace bytes attn_kv4_chunk_fwd needs (kla_attn_kv4_chunk_workspace_bytes)."""
    f, max_len = lib().kla_attn_kv4_chunk_workspace_bytes, min(int(max_len), _INT32)
    if cu_seqlens_host is not None:
        cu = cu_seqlens_host.to("cpu", torch.int32).contiguous()
        # the device pointer is only tested for NULL here
        return f(ctypes.c_void_p(16), cu.data_ptr(), cu.numel() - 1, B, Hq, Hkv, T, D, max_len, _DTYPES[dtype])
    return f(None, None, B, B, Hq, Hkv, T, D, max_len, _DTYPES[dtype])


def attn_kv4_chunk_fwd(
    q: torch.Tensor,
    codes: torch.Tensor,
    scales: torch.Tensor,
    block_table: torch.Tensor,
    seq_lens: torch.Tensor,
    cu_seqlens: Optional[torch.Tensor] = None,
    scale: Optional[float] = None,
    max_len: Optional[int] = None,
    cu_seqlens_host: Optional[torch.Tensor] = None,
    out: Optional[torch.Tensor] = None,
    lse: Optional[torch.Tensor] = None,
    workspace: Optional[torch.Tensor] = None,
) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention of each sequence's newest tokens over a 4-bit cache
    (kla_attn_kv4_chunk_fwd), which holds them already.

    q: [B, Hq, T, D], bf16 or fp32; codes, scales, block_table: the cache; seq_lens: int32 [N]
    cached tokens, the new ones among them; cu_seqlens: int32 [N + 1] packs the new tokens of N
    sequences (B must be 1; None: N = B sequences of T); scale: D ** -0.5 when None; max_len: a bound
    on seq_lens known to the host (the block table's room when None).  Returns (o, lse): lse
    [B, Hq, T] fp32, the logarithm of each query's sum.
    """
    dev, N, host, sizes, cache = _chunk_args("attn_kv4_chunk_fwd", q, codes, scales, block_table, seq_lens, cu_seqlens,
                                             cu_seqlens_host, max_len)
    _, B, Hq, Hkv, T, D = sizes
    if out is None:
        out = torch.empty_like(q)
    else:
        _fit(out, "out", q.dtype, q.shape, dev)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
    else:
        _fit(lse, "lse", torch.float32, (B, Hq, T), dev)
    cu, host_ptr, dt = _ptr(cu_seqlens), _ptr(host), _DTYPES[q.dtype]
    ws = _scratch(workspace, lib().kla_attn_kv4_chunk_workspace_bytes(cu, host_ptr, *sizes, cache[3], dt), dev)
    _call("kla_attn_kv4_chunk_fwd", dev, q.data_ptr(), codes.data_ptr(), scales.data_ptr(), block_table.data_ptr(),
          seq_lens.data_ptr(), D ** -0.5 if scale is None else float(scale), out.data_ptr(), lse.data_ptr(), cu, host_ptr,
          *sizes, *cache, dt, _ptr(ws), 0 if ws is None else ws.numel())
    return out, lse


def kv4_weights(block_table: torch.Tensor, Hkv: int, page_size: int) -> torch.Tensor:
    """No attention weight yet for any token of a cache: zeros [N, Hkv, max_pages * page_size] fp32."""
    N, M = _rank(block_table, "block_table", 2)
    return torch.zeros(N, Hkv, M * page_size, dtype=torch.float32, device=block_table.device)


def attn_kv4_weigh(
    q: torch.Tensor,
    lse: torch.Tensor,
    codes: torch.Tensor,
    scales: torch.Tensor,
    block_table: torch.Tensor,
    seq_lens: torch.Tensor,
    weights: torch.Tensor,
    cu_seqlens: Optional[torch.Tensor] = None,
    scale: Optional[float] = None,
    max_len: Optional[int] = None,
    cu_seqlens_host: Optional[torch.Tensor] = None,
) -> None:
    """Add the attention weight that each sequence's newest tokens give to every cached token
    (kla_attn_kv4_weigh) to ``weights`` [N, Hkv, max_tokens] fp32, in place (kv4_weights makes
    them).  q, lse and the rest as attn_kv4_chunk_fwd's, lse as it returned it."""
    dev, N, host, sizes, cache = _chunk_args("attn_kv4_weigh", q, codes, scales, block_table, seq_lens, cu_seqlens,
                                             cu_seqlens_host, max_len)
    _, B, Hq, Hkv, T, D = sizes
    _fit(lse, "lse", torch.float32, (B, Hq, T), dev)
    W = _rank(weights, "weights", 3)[2]
    _fit(weights, "weights", torch.float32, (N, Hkv, W), dev)
    if W < cache[1] * cache[2]:
        raise ValueError(f"weights has room for {W} tokens, the block table for {cache[1] * cache[2]}")
    _call("kla_attn_kv4_weigh", dev, q.data_ptr(), lse.data_ptr(), codes.data_ptr(), scales.data_ptr(),
          block_table.data_ptr(), seq_lens.data_ptr(), D ** -0.5 if scale is None else float(scale), weights.data_ptr(),
          _ptr(cu_seqlens), _ptr(host), *sizes, *cache, W, _DTYPES[q.dtype])


def kv4_evict_workspace_bytes(N: int, Hkv: int, D: int, budget: int, page_size: int, max_pages: int) -> int:
    """Workspace bytes kv4_evict needs (kla_kv4_evict_workspace_bytes); 0 where the budget covers all
    that the block table has room for."""
    return lib().kla_kv4_evict_workspace_bytes(N, Hkv, D, min(int(budget), _INT32), page_size, max_pages)


def kv4_evict(
    codes: torch.Tensor,
    scales: torch.Tensor,
    block_table: torch.Tensor,
    seq_lens: torch.Tensor,
    weights: torch.Tensor,
    budget: int,
    recent: int = 0,
    workspace: Optional[torch.Tensor] = None,
) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cut every sequence of a 4-bit cache that holds more than ``budget`` tokens to that many
    (kla_kv4_evict), in place, ``weights`` [N, Hkv, max_tokens] too: per key head the newest
    ``recent`` tokens stay and those of the largest weight, in their order.

    Returns (new_lens, kept): int32 [N] cached tokens and int32 [N, Hkv, budget] the former
    position of each token that stays (-1 behind a shorter sequence's).
    """
    if not isinstance(codes, torch.Tensor) or codes.device.type != "cuda":
        raise ValueError("kla.kv4_evict needs GPU tensors")
    dev, N = codes.device, _rank(seq_lens, "seq_lens", 1)[0]
    P, Hkv, page, D, M = _cache_args(codes, scales, block_table, N, dev)
    _fit(seq_lens, "seq_lens", torch.int32, (N,), dev)
    W = _rank(weights, "weights", 3)[2]
    _fit(weights, "weights", torch.float32, (N, Hkv, W), dev)
    if W < M * page:
        raise ValueError(f"weights has room for {W} tokens, the block table for {M * page}")
    budget, recent = int(budget), int(recent)
    if not 1 <= budget <= _MAX_LEN or not 0 <= recent <= budget:
        raise ValueError(f"budget {budget} and recent {recent}: expected 1 <= budget and 0 <= recent <= budget")
    new_lens = torch.empty_like(seq_lens)
    kept = torch.empty((N, Hkv, budget), dtype=torch.int32, device=dev)
    ws = _scratch(workspace, lib().kla_kv4_evict_workspace_bytes(N, Hkv, D, budget, page, M), dev)
    _call("kla_kv4_evict", dev, codes.data_ptr(), scales.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
          weights.data_ptr(), new_lens.data_ptr(), kept.data_ptr(), budget, recent, N, Hkv, D, P, page, M, W, _ptr(ws),
          0 if ws is None else ws.numel())
    return new_lens, kept
