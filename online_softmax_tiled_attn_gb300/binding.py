"""ctypes binding of libosmattn.so: the same entry points as include/osm_attn.h.

Argument marshalling only: every step of the computation runs in the CUDA library.  PyTorch is
used for device memory and streams.  There is no fallback: if the library cannot be built or
loaded, or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

from . import build_lib

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_TIMEOUT = 4
FA_ERR_SCRATCH_LIMIT = 5
FA_ERR_PAGE = 6

OSM_BF16, OSM_FP32 = 0, 1
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3}
KV_FORMATS = {"bf16": 0, "int4": 1}

_lock = threading.Lock()
_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """Load libosmattn.so (building it in-tree with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = build_lib.LIB
            if not build_lib.up_to_date():
                path = build_lib.build()
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library {path} is missing")
            L = ctypes.CDLL(path)
            vp, i64 = ctypes.c_void_p, ctypes.c_int64
            L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float,
                                 ctypes.c_int, vp]
            L.fa_fwd.restype = ctypes.c_int
            L.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64,
                                      i64, ctypes.c_float, ctypes.c_int, i64, vp]
            L.fa_fwd_host.restype = ctypes.c_int
            L.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                         ctypes.c_float, ctypes.c_int, i64, vp, vp, vp]
            L.fa_fwd_splitkv.restype = ctypes.c_int
            L.fa_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                                 ctypes.c_float, ctypes.c_int, i64, vp]
            L.fa_fwd_splitkv_noalloc.restype = ctypes.c_int
            L.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                     ctypes.c_float, ctypes.c_int, vp, i64, vp, vp, vp]
            L.fa_fwd_gqa.restype = ctypes.c_int
            L.fa_fwd_gqa_plan.argtypes = [i64, i64, i64, i64, i64, i64, i64,
                                          ctypes.POINTER(ctypes.c_int64),
                                          ctypes.POINTER(ctypes.c_int64),
                                          ctypes.POINTER(ctypes.c_int64)]
            L.fa_fwd_gqa_plan.restype = ctypes.c_int
            i64p = ctypes.POINTER(ctypes.c_int64)
            L.fa_fwd_splitkv_plan.argtypes = [i64, i64, i64, i64, i64, i64, i64p, i64p, i64p]
            L.fa_fwd_splitkv_plan.restype = ctypes.c_int
            L.osm_softmax.argtypes = [vp, vp, i64, i64, vp, vp]
            L.osm_softmax.restype = ctypes.c_int
            L.fa_fwd_mask.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                      ctypes.c_float, ctypes.c_int, vp, i64, i64, vp, i64, vp]
            L.fa_fwd_mask.restype = ctypes.c_int
            L.fa_fwd_mask_plan.argtypes = [i64, i64, i64, i64, i64, i64, i64p]
            L.fa_fwd_mask_plan.restype = ctypes.c_int
            L.fa_fwd_gqa_mask.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                          ctypes.c_float, ctypes.c_int, vp, vp, i64, i64, vp, i64,
                                          i64, vp, vp, vp]
            L.fa_fwd_gqa_mask.restype = ctypes.c_int
            L.fa_fwd_gqa_mask_plan.argtypes = [i64, i64, i64, i64, i64, i64, i64, i64, i64, i64p,
                                               i64p, i64p, i64p]
            L.fa_fwd_gqa_mask_plan.restype = ctypes.c_int
            L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                 ctypes.c_float, ctypes.c_int, vp]
            L.fa_bwd.restype = ctypes.c_int
            L.fa_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                     i64, ctypes.c_float, ctypes.c_int, vp, vp]
            L.fa_bwd_gqa.restype = ctypes.c_int
            L.osm_softmax_topk.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp]
            L.osm_softmax_topk.restype = ctypes.c_int
            f64, f32, i32 = ctypes.c_double, ctypes.c_float, ctypes.c_int
            L.osm_rope_rates.argtypes = [i64, f64, i32, f64, f64, f64, f64, ctypes.POINTER(f64)]
            L.osm_rope_table.argtypes = [ctypes.POINTER(f64), i64, i64p]
            L.osm_rope.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64p, i64p, vp, i64, vp, i64,
                                   i32, f32, vp]
            L.osm_rope_bwd.argtypes = L.osm_rope.argtypes
            L.osm_kv_page_bytes.argtypes = [i32, i64, i64, i64p]
            L.osm_kv_append.argtypes = [vp, vp, i64p, i64p, vp, vp, i32, i64, i64, vp, i64, vp, vp,
                                        vp, i64, i32, f32, vp, vp, i64p, i64, i64, i64, i64, i64,
                                        vp]
            L.osm_kv_gather.argtypes = [vp, vp, i32, i64, i64, vp, i64, vp, vp, vp, i64, i64, i64,
                                        i64, vp]
            L.fa_fwd_paged.argtypes = [vp, vp, vp, i32, i64, i64, vp, i64, vp, vp, vp, vp, i64, i64,
                                       i64, i64, i64, f32, i32, vp, i64, vp]
            L.fa_fwd_paged_plan.argtypes = [i64, i64, i64, i64, i64, i32, i64, i64, i64p]
            for f in (L.osm_rope_rates, L.osm_rope_table, L.osm_rope, L.osm_rope_bwd,
                      L.osm_kv_page_bytes, L.osm_kv_append, L.osm_kv_gather, L.fa_fwd_paged,
                      L.fa_fwd_paged_plan):
                f.restype = ctypes.c_int
            L.fa_status_string.argtypes = [ctypes.c_int]
            L.fa_status_string.restype = ctypes.c_char_p
            L.osm_attn_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
            L.osm_attn_device_status.restype = ctypes.c_int
            L.osm_attn_selftest_wait.argtypes = [i64, vp]
            L.osm_attn_selftest_wait.restype = ctypes.c_int
            L.osm_attn_abi_version.argtypes = []
            L.osm_attn_abi_version.restype = ctypes.c_int
            _lib = L
        return _lib


def status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


# ------------------------------------------------------------------------------------------
# raw entry points (integers for pointers): the C ABI as is
# ------------------------------------------------------------------------------------------
def fa_fwd_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, N, d, scale, causal, stream_ptr):
    return lib().fa_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, int(B), int(H), int(N), int(d),
                        float(scale), int(bool(causal)), stream_ptr)


def fa_fwd_host_raw(qh, kh, vh, oh, lseh, qd, kd, vd, od, lsed, B, H, N, d, scale, causal,
                    n_chunks, stream_ptr):
    return lib().fa_fwd_host(qh, kh, vh, oh, lseh, qd, kd, vd, od, lsed, int(B), int(H),
                             int(N), int(d), float(scale), int(bool(causal)), int(n_chunks),
                             stream_ptr)


def fa_fwd_splitkv_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nk, d, scale, causal,
                       n_splits, ws_o_ptr, ws_lse_ptr, stream_ptr):
    return lib().fa_fwd_splitkv(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, int(B), int(H), int(Nq),
                                int(Nk), int(d), float(scale), int(bool(causal)), int(n_splits),
                                ws_o_ptr, ws_lse_ptr, stream_ptr)


def fa_fwd_gqa_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, H_kv, Nq, Nk, d, scale, causal,
                   kv_lens_ptr, n_splits, ws_o_ptr, ws_lse_ptr, stream_ptr):
    return lib().fa_fwd_gqa(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, int(B), int(H), int(H_kv),
                            int(Nq), int(Nk), int(d), float(scale), int(bool(causal)),
                            kv_lens_ptr, int(n_splits), ws_o_ptr, ws_lse_ptr, stream_ptr)


def fa_fwd_splitkv_noalloc_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nk, d, scale,
                               causal, n_splits, stream_ptr):
    """The split-key attention with its partial states in the library's fixed scratch array
    (no workspace argument, no allocation)."""
    return lib().fa_fwd_splitkv_noalloc(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, int(B), int(H),
                                        int(Nq), int(Nk), int(d), float(scale),
                                        int(bool(causal)), int(n_splits), stream_ptr)


def splitkv_plan(B, H, Nq, Nk, d, n_splits=0):
    """(splits, workspace O floats, workspace LSE floats) for fa_fwd_splitkv."""
    s, wo, wl = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int64(0)
    rc = lib().fa_fwd_splitkv_plan(int(B), int(H), int(Nq), int(Nk), int(d), int(n_splits),
                                   ctypes.byref(s), ctypes.byref(wo), ctypes.byref(wl))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_splitkv_plan")
    return s.value, wo.value, wl.value


def gqa_plan(B, H, H_kv, Nq, Nk, d, n_splits=0):
    """(splits, workspace O floats, workspace LSE floats) for fa_fwd_gqa."""
    s, wo, wl = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int64(0)
    rc = lib().fa_fwd_gqa_plan(int(B), int(H), int(H_kv), int(Nq), int(Nk), int(d),
                               int(n_splits), ctypes.byref(s), ctypes.byref(wo), ctypes.byref(wl))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_gqa_plan")
    return s.value, wo.value, wl.value


def osm_softmax_raw(x_ptr, y_ptr, rows, cols, lse_ptr, stream_ptr):
    return lib().osm_softmax(x_ptr, y_ptr, int(rows), int(cols), lse_ptr, stream_ptr)


def fa_fwd_mask_raw(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, mask, mask_b_stride,
                    mask_h_stride, tile_map, tile_map_words, stream_ptr):
    return lib().fa_fwd_mask(q, k, v, o, lse, int(B), int(H), int(Nq), int(Nk), int(d),
                             float(scale), int(bool(causal)), mask, int(mask_b_stride),
                             int(mask_h_stride), tile_map, int(tile_map_words), stream_ptr)


def gqa_mask_plan(B, H, H_kv, Nq, Nk, d, mask_b_stride, mask_h_stride, n_splits=0):
    """(splits, workspace O floats, workspace LSE floats, tile map words) for fa_fwd_gqa_mask."""
    s, wo, wl, tm = (ctypes.c_int64(0) for _ in range(4))
    rc = lib().fa_fwd_gqa_mask_plan(int(B), int(H), int(H_kv), int(Nq), int(Nk), int(d),
                                    int(mask_b_stride), int(mask_h_stride), int(n_splits),
                                    ctypes.byref(s), ctypes.byref(wo), ctypes.byref(wl),
                                    ctypes.byref(tm))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_gqa_mask_plan")
    return s.value, wo.value, wl.value, tm.value


def fa_fwd_gqa_mask_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, H_kv, Nq, Nk, d, scale,
                        causal, kv_lens_ptr, mask_ptr, mask_b_stride, mask_h_stride, tm_ptr,
                        tm_words, n_splits, ws_o_ptr, ws_lse_ptr, stream_ptr):
    return lib().fa_fwd_gqa_mask(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, int(B), int(H), int(H_kv),
                                 int(Nq), int(Nk), int(d), float(scale), int(bool(causal)),
                                 kv_lens_ptr, mask_ptr, int(mask_b_stride), int(mask_h_stride),
                                 tm_ptr, int(tm_words), int(n_splits), ws_o_ptr, ws_lse_ptr,
                                 stream_ptr)


def mask_plan(B, H, Nq, Nk, mask_b_stride, mask_h_stride):
    """Words of fa_fwd_mask's tile map for this shape and these mask strides."""
    w = ctypes.c_int64(0)
    rc = lib().fa_fwd_mask_plan(int(B), int(H), int(Nq), int(Nk), int(mask_b_stride),
                                int(mask_h_stride), ctypes.byref(w))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_mask_plan")
    return w.value


def fa_bwd_raw(q, k, v, o, do, lse, dq, dk, dv, ws_d, B, H, N, d, scale, causal, stream_ptr):
    return lib().fa_bwd(q, k, v, o, do, lse, dq, dk, dv, ws_d, int(B), int(H), int(N), int(d),
                        float(scale), int(bool(causal)), stream_ptr)


def osm_softmax_topk_raw(x_ptr, rows, cols, k, values_ptr, indices_ptr, lse_ptr, stream_ptr):
    return lib().osm_softmax_topk(x_ptr, int(rows), int(cols), int(k), values_ptr, indices_ptr,
                                  lse_ptr, stream_ptr)


def selftest_wait(timeout_us: int, stream=None) -> None:
    """Launch the bounded-wait diagnostic (a wait that nothing completes gives up after
    timeout_us and records FA_ERR_TIMEOUT for device_status to report)."""
    rc = lib().osm_attn_selftest_wait(int(timeout_us), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "osm_attn_selftest_wait")


def device_status(stream=None) -> int:
    """Synchronise `stream` and read/clear the kernels' bounded-wait status word."""
    st = ctypes.c_int(0)
    rc = lib().osm_attn_device_status(_stream_handle(stream), ctypes.byref(st))
    if rc != FA_OK:
        raise FaError(rc, "osm_attn_device_status")
    return st.value


# ------------------------------------------------------------------------------------------
# torch-tensor wrappers
# ------------------------------------------------------------------------------------------
def fa_fwd(q, k, v, scale=None, causal=False, out=None, lse=None, return_lse=True,
           stream=None):
    """O, LSE = attention(q, k, v) for CUDA bf16 tensors [B, H, N, d] (d = 64 or 128).

    scale defaults to 1/sqrt(d).  `out` ([B,H,N,d] bf16) and `lse` ([B,H,N] fp32) may be
    given to write into; with return_lse=False and no `lse`, LSE is not computed.
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
    if q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k and v must share one [B, H, N, d] shape")
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise TypeError("out must be a contiguous bf16 tensor shaped like q")
    if lse is None and return_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or lse.numel() != B * H * N
                            or not lse.is_contiguous()):
        raise TypeError("lse must be a contiguous fp32 tensor of B*H*N elements")
    rc = fa_fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                    lse.data_ptr() if lse is not None else None, B, H, N, d, scale, causal,
                    _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd")
    return out, lse


def fa_fwd_host(q, k, v, scale=None, causal=False, out=None, lse=None, return_lse=True,
                staging=None, n_chunks=0, stream=None):
    """O, LSE = attention(q, k, v) for host (CPU) bf16 tensors [B, H, N, d]: the library copies
    groups of heads to the device, runs the attention and copies O and LSE back, the copies
    overlapped with the attention.  q, k, v and `out`/`lse` (host, made page-locked here when
    not given) should be page-locked for the overlap.  `staging` may be the device tensors
    (q_dev, k_dev, v_dev, o_dev, lse_dev or None); otherwise they are allocated here on the
    current CUDA device.  Enqueued on `stream` (the current stream by default); the results are
    ready once it is synchronised, which this function does before it returns."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.is_cuda:
            raise TypeError(f"{name} must be a host (CPU) tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
    if q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k and v must share one [B, H, N, d] shape")
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    if lse is None and return_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32).pin_memory()
    for name, t, dt, n in (("out", out, torch.bfloat16, q.numel()),
                           ("lse", lse, torch.float32, B * H * N)):
        if t is not None and (t.is_cuda or t.dtype != dt or t.numel() != n
                              or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous host tensor of {n} {dt} elements")
    if staging is None:
        dev = torch.device("cuda", torch.cuda.current_device())
        qd = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        staging = (qd, torch.empty_like(qd), torch.empty_like(qd), torch.empty_like(qd),
                   torch.empty((B, H, N), dtype=torch.float32, device=dev)
                   if lse is not None else None)
    qd, kd, vd, od, ld = staging
    for t in (qd, kd, vd, od):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.numel() != q.numel():
            raise TypeError("staging must hold four CUDA bf16 tensors shaped like q")
    if (ld is None) != (lse is None):
        raise TypeError("staging's LSE tensor must be given exactly when lse is")
    s = _stream_handle(stream)
    rc = fa_fwd_host_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                         lse.data_ptr() if lse is not None else None, qd.data_ptr(),
                         kd.data_ptr(), vd.data_ptr(), od.data_ptr(),
                         ld.data_ptr() if ld is not None else None, B, H, N, d, scale, causal,
                         n_chunks, s)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_host")
    (stream if stream is not None else torch.cuda.current_stream()).synchronize()
    return out, lse


def fa_fwd_splitkv(q, k, v, n_splits=0, scale=None, causal=False, out=None, lse=None,
                   return_lse=True, workspace=None, stream=None):
    """Attention of q [B,H,Nq,d] against k, v [B,H,Nk,d] (CUDA bf16) with the keys split into
    key ranges computed in parallel and combined (Flash-Decoding).  n_splits = 0 lets the
    library choose.  `workspace` may be a (ws_O, ws_LSE) pair of fp32 CUDA tensors; otherwise
    it is allocated here (the library itself never allocates).  Returns (O, LSE)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
    if k.shape != v.shape or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("q [B,H,Nq,d] and k, v [B,H,Nk,d] disagree")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    splits, wo, wl = splitkv_plan(B, H, Nq, Nk, d, n_splits)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    ws_o = ws_l = None
    if splits > 1:
        if workspace is None:
            ws_o = torch.empty(wo, dtype=torch.float32, device=q.device)
            ws_l = torch.empty(wl, dtype=torch.float32, device=q.device)
        else:
            ws_o, ws_l = workspace
            if ws_o.numel() < wo or ws_l.numel() < wl:
                raise ValueError("workspace too small for this split count")
    rc = fa_fwd_splitkv_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            lse.data_ptr() if lse is not None else None, B, H, Nq, Nk, d, scale,
                            causal, max(splits, 1) if Nk > 0 else 0,
                            ws_o.data_ptr() if ws_o is not None else None,
                            ws_l.data_ptr() if ws_l is not None else None, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_splitkv")
    return out, lse


def fa_fwd_gqa(q, k, v, kv_lens=None, n_splits=1, scale=None, causal=False, out=None, lse=None,
               return_lse=True, workspace=None, stream=None):
    """Attention of q [B,H,Nq,d] against k, v [B,H_kv,Nk,d] (CUDA bf16; H_kv divides H, query
    head h reads key/value head h // (H // H_kv)), with optional per-sequence key lengths
    kv_lens (CUDA int32 [B]: keys at or past kv_lens[b] are masked).  n_splits = 1 runs one
    pass; 0 lets the library choose a key split (Flash-Decoding), with a workspace allocated
    here unless `workspace` = (ws_O, ws_LSE) is given.  Returns (O, LSE)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
    if k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError("q [B,H,Nq,d] and k, v [B,H_kv,Nk,d] disagree")
    B, H, Nq, d = q.shape
    H_kv, Nk = k.shape[1], k.shape[2]
    if kv_lens is not None:
        if not isinstance(kv_lens, torch.Tensor) or not kv_lens.is_cuda or \
                kv_lens.dtype != torch.int32 or kv_lens.shape != (B,) or \
                not kv_lens.is_contiguous():
            raise TypeError("kv_lens must be a contiguous CUDA int32 tensor of shape [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    splits, wo, wl = gqa_plan(B, H, H_kv, Nq, Nk, d, n_splits)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    ws_o = ws_l = None
    if splits > 1:
        if workspace is None:
            ws_o = torch.empty(wo, dtype=torch.float32, device=q.device)
            ws_l = torch.empty(wl, dtype=torch.float32, device=q.device)
        else:
            ws_o, ws_l = workspace
            if ws_o.numel() < wo or ws_l.numel() < wl:
                raise ValueError("workspace too small for this split count")
    rc = fa_fwd_gqa_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                        lse.data_ptr() if lse is not None else None, B, H, H_kv, Nq, Nk, d, scale,
                        causal, kv_lens.data_ptr() if kv_lens is not None else None,
                        max(splits, 1) if Nk > 0 else 0,
                        ws_o.data_ptr() if ws_o is not None else None,
                        ws_l.data_ptr() if ws_l is not None else None, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_gqa")
    return out, lse


def osm_softmax(x, out=None, lse=None, return_lse=True, stream=None):
    """y, lse = softmax of every row of a CUDA fp32 tensor [rows, cols] (out may be x)."""
    import torch

    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float32:
        raise TypeError("x must be a CUDA fp32 tensor")
    if x.dim() != 2 or not x.is_contiguous():
        raise TypeError("x must be a contiguous [rows, cols] tensor")
    rows, cols = x.shape
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != torch.float32 or not out.is_contiguous():
        raise TypeError("out must be a contiguous fp32 tensor shaped like x")
    if lse is None and return_lse:
        lse = torch.empty((rows,), dtype=torch.float32, device=x.device)
    rc = osm_softmax_raw(x.data_ptr(), out.data_ptr(), rows, cols,
                         lse.data_ptr() if lse is not None else None, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "osm_softmax")
    return out, lse


def osm_softmax_topk(x, k, values=None, indices=None, lse=None, return_lse=True, stream=None):
    """(values, indices, lse): the k largest entries of every row of a CUDA fp32 [rows, cols]
    tensor in descending order (ties: the smaller column first), their softmax shares (fp32)
    and columns (int32), and the rows' log-sum-exp."""
    import torch

    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float32:
        raise TypeError("x must be a CUDA fp32 tensor")
    if x.dim() != 2 or not x.is_contiguous():
        raise TypeError("x must be a contiguous [rows, cols] tensor")
    rows, cols = x.shape
    if values is None:
        values = torch.empty((rows, k), dtype=torch.float32, device=x.device)
    if indices is None:
        indices = torch.empty((rows, k), dtype=torch.int32, device=x.device)
    if lse is None and return_lse:
        lse = torch.empty((rows,), dtype=torch.float32, device=x.device)
    rc = osm_softmax_topk_raw(x.data_ptr(), rows, cols, k, values.data_ptr(), indices.data_ptr(),
                              lse.data_ptr() if lse is not None else None, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "osm_softmax_topk")
    return values, indices, lse


def fa_bwd(q, k, v, o, do, lse, scale=None, causal=False, workspace=None, stream=None):
    """(dQ, dK, dV) of fa_fwd's attention for the output gradient do (CUDA bf16 [B,H,N,d]),
    given the forward's o and lse.  `workspace` may be an fp32 CUDA tensor of B*H*N floats;
    otherwise it is allocated here (the library never allocates)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
        if t.shape != q.shape:
            raise ValueError("q, k, v, o, do must share one shape")
    B, H, N, d = q.shape
    if lse.dtype != torch.float32 or lse.shape != (B, H, N) or not lse.is_contiguous():
        raise TypeError("lse must be a contiguous fp32 [B, H, N] tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    ws_d = (torch.empty(B * H * N, dtype=torch.float32, device=q.device) if workspace is None
            else workspace)
    rc = fa_bwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                    lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws_d.data_ptr(),
                    B, H, N, d, scale, causal, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd")
    return dq, dk, dv


def fa_bwd_gqa_raw(q_ptr, k_ptr, v_ptr, o_ptr, do_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr, ws_ptr,
                   B, H, H_kv, N, d, scale, causal, kv_lens_ptr, stream_ptr):
    return lib().fa_bwd_gqa(q_ptr, k_ptr, v_ptr, o_ptr, do_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr,
                            ws_ptr, int(B), int(H), int(H_kv), int(N), int(d), float(scale),
                            int(bool(causal)), kv_lens_ptr, stream_ptr)


def fa_bwd_gqa(q, k, v, o, do, lse, kv_lens=None, scale=None, causal=False, workspace=None,
               stream=None):
    """(dQ, dK, dV) of fa_fwd_gqa's attention for the output gradient do: q, o, do CUDA bf16
    [B,H,N,d], k, v [B,H_kv,N,d], lse fp32 [B,H,N], optional kv_lens CUDA int32 [B].  dK, dV
    are [B,H_kv,N,d] (a shared key/value head's gradients sum over its query heads)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
    B, H, N, d = q.shape
    H_kv = k.shape[1]
    if o.shape != q.shape or do.shape != q.shape or k.shape != (B, H_kv, N, d) \
            or v.shape != k.shape:
        raise ValueError("q, o, do must be [B, H, N, d] and k, v [B, H_kv, N, d]")
    if lse.dtype != torch.float32 or lse.shape != (B, H, N) or not lse.is_contiguous():
        raise TypeError("lse must be a contiguous fp32 [B, H, N] tensor")
    if kv_lens is not None and (not isinstance(kv_lens, torch.Tensor) or not kv_lens.is_cuda
                                or kv_lens.dtype != torch.int32 or kv_lens.shape != (B,)):
        raise TypeError("kv_lens must be a CUDA int32 [B] tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    ws_d = (torch.empty(B * H * N, dtype=torch.float32, device=q.device) if workspace is None
            else workspace)
    rc = fa_bwd_gqa_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                        lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                        ws_d.data_ptr(), B, H, H_kv, N, d, scale, causal,
                        kv_lens.data_ptr() if kv_lens is not None else None,
                        _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_gqa")
    return dq, dk, dv


def fa_fwd_mask(q, k, v, mask_bits, scale=None, causal=False, out=None, lse=None, stream=None,
                skip_tiles=True, tile_map=None):
    """Attention of q [B,H,Nq,d] over k, v [B,H,Nk,d] (CUDA bf16) with an explicit mask:
    mask_bits is the CUDA uint32/int32 tensor [B or 1, H or 1, Nq, 4 * ceil(Nk / 128)] that
    inputs.pack_mask builds (size-1 leading dimensions repeat).  skip_tiles: pass a tile map
    (tile_map, a CUDA int32 tensor of at least mask_plan words, or one made here) so that key
    tiles with no allowed key are skipped.  Returns (O, LSE)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != k.shape:
        raise ValueError("k, v must be [B, H, Nk, d] with q's B, H and d")
    W = 4 * ((Nk + 127) // 128)
    if (not isinstance(mask_bits, torch.Tensor) or not mask_bits.is_cuda
            or mask_bits.dtype not in (torch.int32, torch.uint32) or mask_bits.dim() != 4
            or not mask_bits.is_contiguous() or tuple(mask_bits.shape[2:]) != (Nq, W)
            or mask_bits.shape[0] not in (1, B) or mask_bits.shape[1] not in (1, H)):
        raise TypeError("mask_bits must be a contiguous CUDA int32 [B or 1, H or 1, Nq, W]")
    hs = Nq * W if mask_bits.shape[1] == H and H > 1 else 0
    bs = mask_bits.shape[1] * Nq * W if mask_bits.shape[0] == B and B > 1 else 0
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    O = torch.empty_like(q) if out is None else out
    L = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    tm_ptr, tm_words = 0, 0
    if skip_tiles:
        need = mask_plan(B, H, Nq, Nk, bs, hs)
        if tile_map is None:
            tile_map = torch.empty(max(need, 1), dtype=torch.int32, device=q.device)
        if (not isinstance(tile_map, torch.Tensor) or not tile_map.is_cuda
                or tile_map.dtype not in (torch.int32, torch.uint32)
                or not tile_map.is_contiguous() or tile_map.numel() < need):
            raise TypeError(f"tile_map must be a contiguous CUDA int32 tensor of >= {need} words")
        tm_ptr, tm_words = tile_map.data_ptr(), tile_map.numel()
    rc = fa_fwd_mask_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), O.data_ptr(), L.data_ptr(),
                         B, H, Nq, Nk, d, scale, causal, mask_bits.data_ptr(), bs, hs,
                         tm_ptr, tm_words, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_mask")
    return O, L


def fa_fwd_gqa_mask(q, k, v, mask_bits, kv_lens=None, n_splits=0, scale=None, causal=False,
                    out=None, lse=None, stream=None, skip_tiles=True, tile_map=None,
                    workspace=None):
    """Attention of q [B,H,Nq,d] over k, v [B,H_kv,Nk,d] (CUDA bf16, H_kv divides H) with an
    explicit mask (mask_bits as for fa_fwd_mask, over the H query heads), optional key lengths
    kv_lens (CUDA int32 [B]) and n_splits key ranges (0: chosen by the plan call; 1: one pass).
    skip_tiles / tile_map as for fa_fwd_mask; workspace: (ws_O, ws_LSE) fp32 CUDA tensors of
    at least the plan's sizes, or made here.  Returns (O, LSE)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 [B, H, N, d] tensor")
    B, H, Nq, d = q.shape
    H_kv, Nk = k.shape[1], k.shape[2]
    if k.shape != (B, H_kv, Nk, d) or v.shape != k.shape:
        raise ValueError("k, v must be [B, H_kv, Nk, d] with q's B and d")
    W = 4 * ((Nk + 127) // 128)
    if (not isinstance(mask_bits, torch.Tensor) or not mask_bits.is_cuda
            or mask_bits.dtype not in (torch.int32, torch.uint32) or mask_bits.dim() != 4
            or not mask_bits.is_contiguous() or tuple(mask_bits.shape[2:]) != (Nq, W)
            or mask_bits.shape[0] not in (1, B) or mask_bits.shape[1] not in (1, H)):
        raise TypeError("mask_bits must be a contiguous CUDA int32 [B or 1, H or 1, Nq, W]")
    if kv_lens is not None and (not isinstance(kv_lens, torch.Tensor) or not kv_lens.is_cuda
                                or kv_lens.dtype != torch.int32 or kv_lens.shape != (B,)):
        raise TypeError("kv_lens must be a CUDA int32 [B] tensor")
    hs = Nq * W if mask_bits.shape[1] == H and H > 1 else 0
    bs = mask_bits.shape[1] * Nq * W if mask_bits.shape[0] == B and B > 1 else 0
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    splits, wo, wl, need = gqa_mask_plan(B, H, H_kv, Nq, Nk, d, bs, hs, n_splits)
    O = torch.empty_like(q) if out is None else out
    L = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    tm_ptr, tm_words = 0, 0
    if skip_tiles:
        if tile_map is None:
            tile_map = torch.empty(max(need, 1), dtype=torch.int32, device=q.device)
        if (not isinstance(tile_map, torch.Tensor) or not tile_map.is_cuda
                or tile_map.dtype not in (torch.int32, torch.uint32)
                or not tile_map.is_contiguous() or tile_map.numel() < need):
            raise TypeError(f"tile_map must be a contiguous CUDA int32 tensor of >= {need} words")
        tm_ptr, tm_words = tile_map.data_ptr(), tile_map.numel()
    ws_o = ws_l = None
    if splits > 1:
        if workspace is None:
            workspace = (torch.empty(wo, dtype=torch.float32, device=q.device),
                         torch.empty(wl, dtype=torch.float32, device=q.device))
        ws_o, ws_l = workspace
        if ws_o.numel() < wo or ws_l.numel() < wl:
            raise ValueError("workspace too small for the plan")
    rc = fa_fwd_gqa_mask_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), O.data_ptr(),
                             L.data_ptr(), B, H, H_kv, Nq, Nk, d, scale, causal,
                             kv_lens.data_ptr() if kv_lens is not None else None,
                             mask_bits.data_ptr(), bs, hs, tm_ptr, tm_words, max(splits, 1),
                             ws_o.data_ptr() if ws_o is not None else None,
                             ws_l.data_ptr() if ws_l is not None else None,
                             _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_gqa_mask")
    return O, L


# ------------------------------------------------------------------------------------------
# rotary positions and the paged key/value cache
# ------------------------------------------------------------------------------------------
_Strides = ctypes.c_int64 * 3


def rope_rates(rot_dim, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, low=1.0,
               high=32.0):
    """The rates (radians a position) of the rot_dim / 2 rotated pairs as a list of floats.
    scaling: "none", "linear", "base" or "bands" (osm_rope_scaling in include/osm_attn.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = (ctypes.c_double * max(1, int(rot_dim) // 2))()
    rc = lib().osm_rope_rates(int(rot_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                              float(orig_len), float(low), float(high), out)
    if rc != FA_OK:
        raise FaError(rc, "osm_rope_rates")
    return list(out)


def rope_table(rates, device="cuda"):
    """The int64 table that the rotating calls take, on `device`, from rates in radians a position
    (rope_rates, or the caller's own).  Made once per model."""
    import torch

    n = len(rates)
    src, out = (ctypes.c_double * max(1, n))(*rates), (ctypes.c_int64 * max(1, n))()
    rc = lib().osm_rope_table(src, n, out)
    if rc != FA_OK:
        raise FaError(rc, "osm_rope_table")
    return torch.tensor(list(out)[:n], dtype=torch.int64).to(device)


# The wrappers below are called once a token and layer: what they check is written for the case that
# passes, and _refuse finds out what was wrong otherwise.
_torch = None


def _load_torch():
    global _torch
    import torch

    _torch = torch
    return torch


def _refuse(t, name, dtype, contiguous):
    torch = _torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    raise TypeError(f"{name} must be a {'contiguous ' if contiguous else ''}{dtype} tensor")


def _ptr(t, name, dtype, dev):
    """Address of a contiguous tensor of this type on the current CUDA device `dev`."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, True)


@functools.lru_cache(maxsize=1024)
def _strides3(b, h, n):
    return _Strides(b, h, n)


def _view(t, name, dtype, dev):
    """(address, strides) of a [B, heads, N, d] tensor whose last dimension is contiguous."""
    try:
        fine = t.dtype is dtype and t.get_device() == dev
    except AttributeError:
        fine = False
    if not fine:
        _refuse(t, name, dtype, False)
    st = t.stride()
    if len(st) != 4:
        raise TypeError(f"{name} must be a [B, heads, N, d] tensor")
    if st[3] != 1 and t.shape[3] > 1:
        raise TypeError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), _strides3(st[0], st[1], st[2])


def _shaped(t, name, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")


def _on(t, name, stream):
    """Index of the current CUDA device and the handle of the stream to launch on, for a call whose
    first tensor is t."""
    torch = _torch or _load_torch()
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = torch.cuda.current_device()
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"stream is on {stream.device}, not on the current CUDA device")
        return dev, int(stream.cuda_stream)
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _empty(shape, dtype, device, stream):
    """A tensor for a call on `stream` (None: the current one), from that stream's memory: memory of
    another stream could still be in use there when the call runs.  The current stream, where the
    result will be used, is recorded with it."""
    torch = _torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _rope_args(table, rot_dim, layout, d, dev):
    lay = ROPE_LAYOUTS.get(layout)
    if lay is None:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    ptr = _ptr(table, "table", _torch.int64, dev)
    ts = table.shape
    rot = 2 * ts[0] if len(ts) == 1 else 0
    if rot < 2 or rot > d or (rot_dim is not None and rot_dim != rot):
        raise ValueError(f"table must hold the rates of rot_dim / 2 pairs, rot_dim at most {d}")
    return ptr, rot, lay


def _rope(call, what, x, table, positions, layout, amplitude, out, rot_dim, stream):
    dev, handle = _on(x, "x", stream)
    torch = _torch
    dtype = x.dtype
    if dtype is torch.bfloat16:
        code = OSM_BF16
    elif dtype is torch.float32:
        code = OSM_FP32
    else:
        raise TypeError("x must be a bf16 or fp32 [B, H, N, d] tensor")
    xp, xs = _view(x, "x", dtype, dev)
    shape = x.shape
    B, H, N, d = shape
    tp, rot, lay = _rope_args(table, rot_dim, layout, d, dev)
    if out is None:
        out = _empty(shape, dtype, x.device, stream)
        op, os_ = out.data_ptr(), _strides3(H * N * d, N * d, d)
    else:
        op, os_ = _view(out, "out", dtype, dev)
        _shaped(out, "out", shape)
    pp, bs = None, 0
    if positions is not None:
        pp = _ptr(positions, "positions", torch.int32, dev)
        ps = positions.shape
        n = len(ps)
        if n == 0 or n > 2 or ps[-1] != N or (n == 2 and ps[0] != 1 and ps[0] != B):
            raise ValueError("positions must be int32 [N], [1, N] or [B, N]")
        if n == 2 and ps[0] > 1:
            bs = N
    rc = call(xp, op, code, B, H, N, d, xs, os_, pp, bs, tp, rot, lay, amplitude, handle)
    if rc != FA_OK:
        raise FaError(rc, what)
    return out


def osm_rope(x, table, positions=None, layout="half", amplitude=1.0, out=None, rot_dim=None,
             stream=None):
    """x (CUDA bf16 or fp32 [B, H, N, d], any strides with d innermost) with the first
    2 * len(table) values of every head rotated by their token's position (positions int32 [N] or
    [B, N]; None: 0 .. N-1).  layout "half" pairs value i with i + rot_dim / 2, "interleaved" 2 i
    with 2 i + 1.  out: made contiguous here unless given; may be x."""
    return _rope(lib().osm_rope, "osm_rope", x, table, positions, layout, amplitude, out, rot_dim,
                 stream)


def osm_rope_bwd(dy, table, positions=None, layout="half", amplitude=1.0, out=None, rot_dim=None,
                 stream=None):
    """The gradient of osm_rope's input from that of its output (arguments as osm_rope's)."""
    return _rope(lib().osm_rope_bwd, "osm_rope_bwd", dy, table, positions, layout, amplitude, out,
                 rot_dim, stream)


def kv_page_bytes(format, page_size, d):
    """Bytes of one key/value head of a page ("bf16" or "int4")."""
    n = ctypes.c_int64(0)
    rc = lib().osm_kv_page_bytes(KV_FORMATS[format], int(page_size), int(d), ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "osm_kv_page_bytes")
    return n.value


def kv_pages(num_pages, H_kv, page_size, d, format="bf16", device="cuda"):
    """(k_pages, v_pages) of an empty cache: bf16 [num_pages, H_kv, page_size, d], or, "int4",
    uint8 [num_pages, H_kv, kv_page_bytes("int4", page_size, d)]."""
    import torch

    n = kv_page_bytes(format, page_size, d)
    shape, dtype = (((num_pages, H_kv, page_size, d), torch.bfloat16) if format == "bf16" else
                    ((num_pages, H_kv, n), torch.uint8))
    return tuple(torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))


def _cache(k_pages, v_pages, page_table, B, H_kv, d, dev):
    """(k, v pointers, format, num_pages, page_size, table pointer, max_pages)."""
    torch = _torch
    bf16 = torch.bfloat16
    fmt = 0 if getattr(k_pages, "dtype", None) is bf16 else 1
    dtype = torch.uint8 if fmt else bf16
    kp = _ptr(k_pages, "k_pages", dtype, dev)
    vp = _ptr(v_pages, "v_pages", dtype, dev)
    shape = k_pages.shape
    _shaped(v_pages, "v_pages", shape)
    if len(shape) != (3 if fmt else 4) or shape[1] != H_kv:
        raise ValueError(f"pages must be bf16 [num_pages, {H_kv}, page_size, d] or uint8 "
                         f"[num_pages, {H_kv}, page bytes]")
    page = shape[2]
    if fmt:
        row = d // 2 + d // 32
        if page % row != 0:
            raise ValueError(f"a 4-bit page head must be a multiple of {row} bytes")
        page //= row
    elif shape[3] != d:
        raise ValueError(f"pages hold heads of {shape[3]} values, not {d}")
    tp = _ptr(page_table, "page_table", torch.int32, dev)
    ts = page_table.shape
    if len(ts) != 2 or ts[0] != B:
        raise ValueError(f"page_table must be int32 [{B}, max_pages]")
    return kp, vp, fmt, shape[0], page, tp, ts[1]


def _heads(pages):
    """Key/value heads of a page array."""
    shape = getattr(pages, "shape", ())
    if len(shape) < 2:
        raise TypeError("k_pages must be a page array (see kv_pages)")
    return shape[1]


def _lens(t, name, B, dev):
    p = _ptr(t, name, _torch.int32, dev)
    ts = t.shape
    if len(ts) != 1 or ts[0] != B:
        raise ValueError(f"{name} must be int32 [{B}]")
    return p


def osm_kv_append(k, v, k_pages, v_pages, page_table, cache_lens, new_lens=None, table=None,
                  layout="half", amplitude=1.0, q=None, q_out=None, stream=None):
    """Writes tokens' keys and values (CUDA bf16 [B, H_kv, N, d], any strides with d innermost)
    into the paged cache: token n < new_lens[b] (int32 [B]; None: all N) at position
    cache_lens[b] + n (int32 [B]), the keys rotated by it when `table` is given.  With q
    ([B, H, N, d]) its rows are rotated into q_out (made here unless given; contiguous).  The pages
    are bf16 or 4-bit by their type (kv_pages).  Returns q_out."""
    dev, handle = _on(k, "k", stream)
    bf16 = _torch.bfloat16
    kp, ks = _view(k, "k", bf16, dev)
    vp, vs = _view(v, "v", bf16, dev)
    shape = k.shape
    _shaped(v, "v", shape)
    B, H_kv, N, d = shape
    cache = _cache(k_pages, v_pages, page_table, B, H_kv, d, dev)
    cl = _lens(cache_lens, "cache_lens", B, dev)
    nl = _lens(new_lens, "new_lens", B, dev) if new_lens is not None else None
    tp, rot, lay = (None, 0, 0) if table is None else _rope_args(table, None, layout, d, dev)
    qp = op = qs = None
    H = 0
    if q is not None:
        qp, qs = _view(q, "q", bf16, dev)
        qshape = q.shape
        H = qshape[1]
        if qshape[0] != B or qshape[2] != N or qshape[3] != d:
            raise ValueError("q must be [B, H, N, d] with k's B, N and d")
        if q_out is None:
            q_out = _empty(qshape, bf16, q.device, stream)
            op = q_out.data_ptr()
        else:
            op = _ptr(q_out, "q_out", bf16, dev)
            _shaped(q_out, "q_out", qshape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = lib().osm_kv_append(kp, vp, ks, vs, *cache, cl, nl, tp, rot, lay, amplitude, qp, op, qs, B,
                             H, H_kv, N, d, handle)
    if rc != FA_OK:
        raise FaError(rc, "osm_kv_append")
    return q_out


def osm_kv_gather(k_pages, v_pages, page_table, kv_lens, N, d, k_out=None, v_out=None,
                  stream=None):
    """(K, V) bf16 [B, H_kv, N, d]: the first kv_lens[b] (int32 [B]) cached tokens of every
    sequence, and zeros behind them."""
    dev, handle = _on(k_pages, "k_pages", stream)
    bf16 = _torch.bfloat16
    H_kv = _heads(k_pages)
    B, N, d = len(page_table), int(N), int(d)
    cache = _cache(k_pages, v_pages, page_table, B, H_kv, d, dev)
    kl = _lens(kv_lens, "kv_lens", B, dev)
    shape = (B, H_kv, N, d)
    if k_out is None:
        k_out = _empty(shape, bf16, k_pages.device, stream)
    if v_out is None:
        v_out = _empty(shape, bf16, k_pages.device, stream)
    kp = _ptr(k_out, "k_out", bf16, dev)
    vp = _ptr(v_out, "v_out", bf16, dev)
    _shaped(k_out, "k_out", shape)
    _shaped(v_out, "v_out", shape)
    rc = lib().osm_kv_gather(*cache, kl, kp, vp, B, H_kv, N, d, handle)
    if rc != FA_OK:
        raise FaError(rc, "osm_kv_gather")
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def _paged_bytes(dev, B, H, H_kv, Nq, d, fmt, page_size, max_pages):
    """fa_fwd_paged_plan for the current device `dev` (its SM count enters)."""
    n = ctypes.c_int64(0)
    rc = lib().fa_fwd_paged_plan(B, H, H_kv, Nq, d, fmt, page_size, max_pages, ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_paged_plan")
    return n.value


def paged_plan(B, H, H_kv, Nq, d, format, page_size, max_pages):
    """Workspace bytes of fa_fwd_paged ("bf16" or "int4" pages) on the current CUDA device."""
    torch = _torch or _load_torch()
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    return _paged_bytes(dev, int(B), int(H), int(H_kv), int(Nq), int(d), KV_FORMATS[format],
                        int(page_size), int(max_pages))


def fa_fwd_paged(q, k_pages, v_pages, page_table, kv_lens, q_lens=None, scale=None, causal=True,
                 out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """Attention of q (CUDA bf16 [B, H, Nq, d]) over a paged cache of kv_lens[b] (int32 [B]) tokens
    a sequence.  Rows i < q_lens[b] (int32 [B]; None: all Nq) are queries; causal: query i is token
    kv_lens[b] - q_lens[b] + i and sees the keys up to itself.  `workspace`: a CUDA tensor of
    paged_plan bytes, made here unless given.  Returns (O, LSE)."""
    dev, handle = _on(q, "q", stream)
    torch = _torch
    bf16 = torch.bfloat16
    qp = _ptr(q, "q", bf16, dev)
    shape = q.shape
    if len(shape) != 4:
        raise TypeError("q must be a bf16 [B, H, Nq, d] tensor")
    B, H, Nq, d = shape
    H_kv = _heads(k_pages)
    cache = _cache(k_pages, v_pages, page_table, B, H_kv, d, dev)
    kl = _lens(kv_lens, "kv_lens", B, dev)
    ql = _lens(q_lens, "q_lens", B, dev) if q_lens is not None else None
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = _paged_bytes(dev, B, H, H_kv, Nq, d, cache[2], cache[4], cache[6])
    device = q.device
    if out is None:
        out = _empty(shape, bf16, device, stream)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", bf16, dev)
        _shaped(out, "out", shape)
    lp = None
    if lse is not None:
        lp = _ptr(lse, "lse", torch.float32, dev)
        _shaped(lse, "lse", (B, H, Nq))
    elif return_lse:
        lse = _empty((B, H, Nq), torch.float32, device, stream)
        lp = lse.data_ptr()
    wp = None
    if workspace is not None:
        wp = _ptr(workspace, "workspace", workspace.dtype, dev)
        if workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace must hold at least {need} bytes")
    elif need > 0:
        workspace = _empty(need, torch.uint8, device, stream)
        wp = workspace.data_ptr()
    rc = lib().fa_fwd_paged(qp, *cache, kl, ql, op, lp, B, H, H_kv, Nq, d, scale, int(bool(causal)),
                            wp, need, handle)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_paged")
    return out, lse
