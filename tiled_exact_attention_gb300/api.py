"""Python entry points with the same names as the C ABI (argument marshalling only).

Tensors are torch CUDA tensors: Q, O ``[b, sq, hq, d]``, K, V ``[b, skv, hkv, d]``
(head dimension contiguous), LSE fp32 ``[b, hq, sq]``.  PyTorch provides the
device memory and the current stream; every step of the computation runs in
libfa.so.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import (FA_BF16, FA_FP16, FA_OFFSET_BOTTOM_RIGHT, KV_APPEND, KV_GATHER_INT4, KVCACHE_INT4, BwdArgs,
                   E4m3Args, FwdArgs, KvcacheArgs, QuantArgs, SplitkvE4m3Args, VarlenArgs, check)

_DT = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


def _strides(t: torch.Tensor):
    s = t.stride()
    return (ctypes.c_int64 * 3)(s[0], s[1], s[2])


def _check_qkv(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be 4-D [b, s, h, d]")
        if t.dtype not in _DT:
            raise ValueError(f"{name} must be bf16 or fp16")
        if t.stride(3) != 1:
            raise ValueError(f"{name} must have a contiguous head dimension")
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError("q, k, v must share a dtype")
    if k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError("inconsistent q/k/v shapes")


def make_args(q, k, v, o, lse, *, causal: bool, scale: float | None, q_pos_offset: int | None,
              window=None, softcap: float = 0.0) -> FwdArgs:
    """Fill `fa_fwd_args`.  window = (left, right) turns on the sliding window (-1 leaves a side open);
    softcap = c > 0 caps every scaled score s to c * tanh(s / c)."""
    _check_qkv(q, k, v)
    b, sq, hq, d = q.shape
    skv, hkv = k.shape[1], k.shape[2]
    a = FwdArgs()
    a.dtype = _DT[q.dtype]
    a.b, a.sq, a.skv, a.hq, a.hkv, a.d = b, sq, skv, hq, hkv, d
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    a.o, a.lse = o.data_ptr(), lse.data_ptr()
    a.q_strides, a.k_strides, a.v_strides, a.o_strides = _strides(q), _strides(k), _strides(v), _strides(o)
    a.causal = 1 if causal else 0
    a.q_pos_offset = FA_OFFSET_BOTTOM_RIGHT if q_pos_offset is None else int(q_pos_offset)
    a.scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    if window is not None:
        a.local = 1
        a.window_left, a.window_right = int(window[0]), int(window[1])
    a.softcap = float(softcap)
    return a


def _outputs(q, out, lse):
    b, sq, hq, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((b, hq, sq), dtype=torch.float32, device=q.device)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_cuda or out.stride(3) != 1:
        raise ValueError("out must match q")
    if lse.shape != (b, hq, sq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [b, hq, sq]")
    return out, lse


def fa_fwd(q, k, v, *, causal: bool = False, scale: float | None = None, q_pos_offset: int | None = None,
           out=None, lse=None, stream=None, window=None, softcap: float = 0.0):
    """Forward pass; returns (O, LSE)."""
    out, lse = _outputs(q, out, lse)
    a = make_args(q, k, v, out, lse, causal=causal, scale=scale, q_pos_offset=q_pos_offset, window=window,
                  softcap=softcap)
    check(_lib.load().fa_fwd(ctypes.byref(a), _stream_handle(stream)), "fa_fwd")
    return out, lse


def fa_num_splits_heuristic(units: int, slots: int, num_kv_blocks: int, max_splits: int = 128) -> int:
    return int(_lib.load().fa_num_splits_heuristic(units, slots, num_kv_blocks, max_splits))


def fa_splitkv_default_splits(q, k, v, *, causal=False, scale=None, q_pos_offset=None, window=None,
                              softcap: float = 0.0) -> int:
    out, lse = _outputs(q, None, None)
    a = make_args(q, k, v, out, lse, causal=causal, scale=scale, q_pos_offset=q_pos_offset, window=window,
                  softcap=softcap)
    return int(_lib.load().fa_splitkv_default_splits(ctypes.byref(a)))


def fa_splitkv_workspace_size(q, k, v, num_splits: int = 0, *, causal=False, scale=None,
                              q_pos_offset=None, window=None, softcap: float = 0.0) -> int:
    out, lse = _outputs(q, None, None)
    a = make_args(q, k, v, out, lse, causal=causal, scale=scale, q_pos_offset=q_pos_offset, window=window,
                  softcap=softcap)
    return int(_lib.load().fa_splitkv_workspace_size(ctypes.byref(a), num_splits))


def fa_fwd_splitkv(q, k, v, *, causal: bool = False, scale: float | None = None, q_pos_offset: int | None = None,
                   num_splits: int = 0, workspace=None, out=None, lse=None, stream=None, return_splits=False,
                   window=None, softcap: float = 0.0):
    """Split-KV forward + combine; returns (O, LSE) (and the split count if asked)."""
    out, lse = _outputs(q, out, lse)
    a = make_args(q, k, v, out, lse, causal=causal, scale=scale, q_pos_offset=q_pos_offset, window=window,
                  softcap=softcap)
    lib = _lib.load()
    need = int(lib.fa_splitkv_workspace_size(ctypes.byref(a), int(num_splits)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    used = ctypes.c_int32(0)
    check(lib.fa_fwd_splitkv(ctypes.byref(a), int(num_splits), ctypes.c_void_p(workspace.data_ptr()),
                             workspace.numel() * workspace.element_size(), ctypes.byref(used),
                             _stream_handle(stream)), "fa_fwd_splitkv")
    if return_splits:
        return out, lse, int(used.value)
    return out, lse


def fa_fwd_splitkv_noalloc(q, k, v, *, causal: bool = False, scale: float | None = None,
                           q_pos_offset: int | None = None, num_splits: int = 0, out=None, lse=None, stream=None,
                           return_splits=False, window=None, softcap: float = 0.0):
    """Split-KV forward that uses the library's built-in scratch instead of a workspace."""
    out, lse = _outputs(q, out, lse)
    a = make_args(q, k, v, out, lse, causal=causal, scale=scale, q_pos_offset=q_pos_offset, window=window,
                  softcap=softcap)
    used = ctypes.c_int32(0)
    check(_lib.load().fa_fwd_splitkv_noalloc(ctypes.byref(a), int(num_splits), ctypes.byref(used),
                                             _stream_handle(stream)), "fa_fwd_splitkv_noalloc")
    if return_splits:
        return out, lse, int(used.value)
    return out, lse


def make_kvcache_args(q, k, v, o, lse, *, block_table=None, seqlens_k=None, cu_seqlens_k=None,
                      max_seqlen_k: int = 0, scale: float | None = None, window_left=None,
                      softcap: float = 0.0) -> KvcacheArgs:
    """Fill `fa_kvcache_args`.  q, o: [b, hq, d]; paged k/v: [num_pages, page_size, hkv, d] with
    block_table [b, n] and seqlens_k [b] (int32); packed k/v: [total_k, hkv, d] with cu_seqlens_k [b + 1].
    window_left (not None) keeps only the last window_left + 1 keys of each sequence."""
    for name, t in (("q", q), ("k", k), ("v", v), ("out", o)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DT or t.stride(-1) != 1:
            raise ValueError(f"{name} must be a CUDA bf16/fp16 tensor with a contiguous last dimension")
    if q.dim() != 3 or o.shape != q.shape:
        raise ValueError("q and out must be [b, hq, d]")
    b, hq, d = q.shape
    a = KvcacheArgs()
    a.dtype = _DT[q.dtype]
    a.b, a.hq, a.d = b, hq, d
    a.q = q.data_ptr()
    a.q_strides = (ctypes.c_int64 * 2)(q.stride(0), q.stride(1))
    a.k, a.v = k.data_ptr(), v.data_ptr()
    if block_table is not None:
        if k.dim() != 4 or v.shape != k.shape or seqlens_k is None:
            raise ValueError("paged cache: k, v [num_pages, page_size, hkv, d] and seqlens_k are required")
        for t in (block_table, seqlens_k):
            if t.dtype != torch.int32 or not t.is_cuda:
                raise ValueError("block_table and seqlens_k must be CUDA int32 tensors")
        a.num_pages, a.page_size, a.hkv = k.shape[0], k.shape[1], k.shape[2]
        a.k_strides = (ctypes.c_int64 * 3)(k.stride(0), k.stride(1), k.stride(2))
        a.v_strides = (ctypes.c_int64 * 3)(v.stride(0), v.stride(1), v.stride(2))
        a.block_table = block_table.data_ptr()
        a.block_table_stride = block_table.stride(0)
        a.seqlens_k = seqlens_k.data_ptr()
    else:
        if k.dim() != 3 or v.shape != k.shape or cu_seqlens_k is None:
            raise ValueError("packed keys: k, v [total_k, hkv, d] and cu_seqlens_k are required")
        if cu_seqlens_k.dtype != torch.int32 or not cu_seqlens_k.is_cuda:
            raise ValueError("cu_seqlens_k must be a CUDA int32 tensor")
        a.num_pages, a.page_size, a.hkv = k.shape[0], 0, k.shape[1]
        a.k_strides = (ctypes.c_int64 * 3)(0, k.stride(0), k.stride(1))
        a.v_strides = (ctypes.c_int64 * 3)(0, v.stride(0), v.stride(1))
        a.cu_seqlens_k = cu_seqlens_k.data_ptr()
    a.max_seqlen_k = int(max_seqlen_k)
    a.o = o.data_ptr()
    a.o_strides = (ctypes.c_int64 * 2)(o.stride(0), o.stride(1))
    a.lse = lse.data_ptr()
    a.scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    if window_left is not None:
        a.local, a.window_left = 1, int(window_left)
    a.softcap = float(softcap)
    return a


def fa_fwd_kvcache(q, k, v, *, block_table=None, seqlens_k=None, cu_seqlens_k=None, max_seqlen_k=None,
                   scale=None, num_splits: int = 0, workspace=None, out=None, lse=None, stream=None,
                   return_splits=False, window_left=None, softcap: float = 0.0):
    """Decode one query row per sequence against a paged or packed KV cache; returns (O [b, hq, d], LSE [b, hq])."""
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if max_seqlen_k is None:
        lens = seqlens_k if block_table is not None else (cu_seqlens_k[1:] - cu_seqlens_k[:-1])
        max_seqlen_k = int(lens.max().item()) if lens.numel() else 0
    a = make_kvcache_args(q, k, v, out, lse, block_table=block_table, seqlens_k=seqlens_k,
                          cu_seqlens_k=cu_seqlens_k, max_seqlen_k=max_seqlen_k, scale=scale,
                          window_left=window_left, softcap=softcap)
    lib = _lib.load()
    if workspace is None:
        need = int(lib.fa_kvcache_workspace_size(ctypes.byref(a), int(num_splits)))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    used = ctypes.c_int32(0)
    check(lib.fa_fwd_kvcache(ctypes.byref(a), int(num_splits), ctypes.c_void_p(workspace.data_ptr()),
                             workspace.numel() * workspace.element_size(), ctypes.byref(used),
                             _stream_handle(stream)), "fa_fwd_kvcache")
    if return_splits:
        return out, lse, int(used.value)
    return out, lse


def make_varlen_args(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int, causal: bool,
                     scale: float | None, window=None, softcap: float = 0.0) -> VarlenArgs:
    """Fill `fa_varlen_args`.  q, o: [total_q, hq, d]; k, v: [total_k, hkv, d]; lse: fp32 [hq, total_q];
    cu_seqlens_q / cu_seqlens_k: CUDA int32 [b + 1] prefix sums."""
    for name, t in (("q", q), ("k", k), ("v", v), ("out", o)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DT or t.dim() != 3 \
                or t.stride(2) != 1:
            raise ValueError(f"{name} must be a CUDA bf16/fp16 [rows, heads, d] tensor with contiguous d")
    if q.dtype != k.dtype or q.dtype != v.dtype or o.dtype != q.dtype:
        raise ValueError("q, k, v, out must share a dtype")
    if k.shape != v.shape or q.shape[2] != k.shape[2] or o.shape != q.shape:
        raise ValueError("inconsistent q/k/v/out shapes")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if t.dtype != torch.int32 or not t.is_cuda or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA int32 vector")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both hold b + 1 >= 2 entries")
    total_q, hq, d = q.shape
    total_k, hkv = k.shape[0], k.shape[1]
    if lse.shape != (hq, total_q) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [hq, total_q]")
    a = VarlenArgs()
    a.dtype = _DT[q.dtype]
    a.b = cu_seqlens_q.numel() - 1
    a.hq, a.hkv, a.d = hq, hkv, d
    a.total_q, a.total_k, a.max_seqlen_q = total_q, total_k, int(max_seqlen_q)
    a.q, a.k, a.v, a.o, a.lse = q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr()
    a.q_strides = (ctypes.c_int64 * 2)(q.stride(0), q.stride(1))
    a.k_strides = (ctypes.c_int64 * 2)(k.stride(0), k.stride(1))
    a.v_strides = (ctypes.c_int64 * 2)(v.stride(0), v.stride(1))
    a.o_strides = (ctypes.c_int64 * 2)(o.stride(0), o.stride(1))
    a.cu_seqlens_q, a.cu_seqlens_k = cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr()
    a.causal = 1 if causal else 0
    if window is not None:
        a.local = 1
        a.window_left, a.window_right = int(window[0]), int(window[1])
    a.scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    a.softcap = float(softcap)
    return a


def fa_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int | None = None, causal: bool = False,
                  scale: float | None = None, window=None, out=None, lse=None, stream=None, softcap: float = 0.0):
    """Forward pass over packed variable-length sequences; returns (O [total_q, hq, d], LSE [hq, total_q]).
    max_seqlen_q defaults to the longest sequence (read back from the device once)."""
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    if max_seqlen_q is None:
        lens = cu_seqlens_q[1:] - cu_seqlens_q[:-1]
        max_seqlen_q = int(lens.max().item()) if lens.numel() else 0
    a = make_varlen_args(q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q, causal=causal,
                         scale=scale, window=window, softcap=softcap)
    check(_lib.load().fa_fwd_varlen(ctypes.byref(a), _stream_handle(stream)), "fa_fwd_varlen")
    return out, lse


def make_bwd_args(q, k, v, o, lse, dout, dq, dk, dv, *, causal: bool, scale: float | None,
                  q_pos_offset: int | None, window=None, softcap: float = 0.0) -> BwdArgs:
    """Fill `fa_bwd_args` from [b, s, h, d] tensors (lse fp32 [b, hq, sq])."""
    _check_qkv(q, k, v)
    for name, t, like in (("o", o, q), ("dout", dout, q), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.shape != like.shape or t.dtype != q.dtype \
                or t.stride(3) != 1:
            raise ValueError(f"{name} must be a CUDA tensor shaped and typed like its forward counterpart")
    b, sq, hq, d = q.shape
    if lse.shape != (b, hq, sq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [b, hq, sq]")
    a = BwdArgs()
    a.dtype = _DT[q.dtype]
    a.b, a.sq, a.skv, a.hq, a.hkv, a.d = b, sq, k.shape[1], hq, k.shape[2], d
    a.q, a.k, a.v, a.o, a.dout, a.lse = (t.data_ptr() for t in (q, k, v, o, dout, lse))
    a.dq, a.dk, a.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    a.q_strides, a.k_strides, a.v_strides = _strides(q), _strides(k), _strides(v)
    a.o_strides, a.do_strides = _strides(o), _strides(dout)
    a.dq_strides, a.dk_strides, a.dv_strides = _strides(dq), _strides(dk), _strides(dv)
    a.causal = 1 if causal else 0
    a.q_pos_offset = FA_OFFSET_BOTTOM_RIGHT if q_pos_offset is None else int(q_pos_offset)
    a.scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    if window is not None:
        a.local = 1
        a.window_left, a.window_right = int(window[0]), int(window[1])
    a.softcap = float(softcap)
    return a


def fa_bwd_workspace_size(q, k, v, *, causal: bool = False, scale: float | None = None,
                          q_pos_offset: int | None = None, window=None, softcap: float = 0.0) -> int:
    """Device workspace bytes fa_bwd needs for these shapes (D and L * log2(e) per padded row)."""
    b, sq, hq, _ = q.shape
    lse = torch.empty((b, hq, sq), dtype=torch.float32, device=q.device)
    a = make_bwd_args(q, k, v, q, lse, q, q, k, v, causal=causal, scale=scale, q_pos_offset=q_pos_offset,
                      window=window, softcap=softcap)
    return int(_lib.load().fa_bwd_workspace_size(ctypes.byref(a)))


def fa_bwd(q, k, v, o, lse, dout, *, causal: bool = False, scale: float | None = None,
           q_pos_offset: int | None = None, window=None, dq=None, dk=None, dv=None, workspace=None, stream=None,
           softcap: float = 0.0):
    """Backward pass for the forward call with the same arguments; returns (dQ, dK, dV)."""
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    a = make_bwd_args(q, k, v, o, lse, dout, dq, dk, dv, causal=causal, scale=scale, q_pos_offset=q_pos_offset,
                      window=window, softcap=softcap)
    lib = _lib.load()
    if workspace is None:
        need = int(lib.fa_bwd_workspace_size(ctypes.byref(a)))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    check(lib.fa_bwd(ctypes.byref(a), ctypes.c_void_p(workspace.data_ptr()),
                     workspace.numel() * workspace.element_size(), _stream_handle(stream)), "fa_bwd")
    return dq, dk, dv


def fa_quantize_e4m3(x, *, per_head: bool = False, transpose: bool = False, stream=None):
    """e4m3 codes (torch.uint8) of a [b, s, h, d] bf16/fp16 tensor and their descales (fp32).
    Codes are [b, s, h, d], or [b, h, d, s_pad] (s_pad = s rounded up to 16) with transpose=True;
    descales are [b, h, ceil(s / 128)] per 128-row block, or [b, h] with per_head=True."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in _DT or x.dim() != 4 or x.stride(3) != 1:
        raise ValueError("x must be a CUDA bf16/fp16 [b, s, h, d] tensor with contiguous d")
    b, s, h, d = x.shape
    if transpose:
        sp = (s + 15) // 16 * 16
        out = torch.zeros((b, h, d, sp), dtype=torch.uint8, device=x.device)
        ost = (out.stride(0), out.stride(1), out.stride(2))
    else:
        out = torch.empty((b, s, h, d), dtype=torch.uint8, device=x.device)
        ost = (out.stride(0), out.stride(1), out.stride(2))
    ds = torch.empty((b, h) if per_head else (b, h, (s + 127) // 128), dtype=torch.float32, device=x.device)
    a = QuantArgs()
    a.dtype = _DT[x.dtype]
    a.b, a.s, a.h, a.d = b, s, h, d
    a.x = x.data_ptr()
    a.x_strides = _strides(x)
    a.out = out.data_ptr()
    a.out_strides = (ctypes.c_int64 * 3)(*ost)
    a.transpose, a.per_head = int(bool(transpose)), int(bool(per_head))
    a.descale = ds.data_ptr()
    check(_lib.load().fa_quantize_e4m3(ctypes.byref(a), _stream_handle(stream)), "fa_quantize_e4m3")
    return out, ds


def quantize_qkv_e4m3(q, k, v, stream=None):
    """The inputs fa_fwd_e4m3 expects: (q8, q_descale), (k8, k_descale) per 128-row block, and V
    transposed with one descale per (batch, head)."""
    return (fa_quantize_e4m3(q, stream=stream), fa_quantize_e4m3(k, stream=stream),
            fa_quantize_e4m3(v, per_head=True, transpose=True, stream=stream))


def fa_fwd_e4m3(q8, q_descale, k8, k_descale, vt8, v_descale, *, causal: bool = False, scale: float | None = None,
                q_pos_offset: int | None = None, window=None, out=None, lse=None, stream=None):
    """Forward pass on e4m3 inputs (see fa_quantize_e4m3); returns (O bf16 [b, sq, hq, d], LSE [b, hq, sq])."""
    for name, t in (("q8", q8), ("k8", k8), ("vt8", vt8)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.uint8 or t.dim() != 4 \
                or t.stride(3) != 1:
            raise ValueError(f"{name} must be a CUDA uint8 4-D tensor with a contiguous last dimension")
    b, sq, hq, d = q8.shape
    skv, hkv = k8.shape[1], k8.shape[2]
    if k8.shape != (b, skv, hkv, d) or vt8.shape[:3] != (b, hkv, d) or vt8.shape[3] < skv:
        raise ValueError("inconsistent q8 / k8 / vt8 shapes")
    if out is None:
        out = torch.empty((b, sq, hq, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((b, hq, sq), dtype=torch.float32, device=q8.device)
    a = E4m3Args()
    a.b, a.sq, a.skv, a.hq, a.hkv, a.d = b, sq, skv, hq, hkv, d
    a.q, a.k, a.vt = q8.data_ptr(), k8.data_ptr(), vt8.data_ptr()
    a.q_descale, a.k_descale, a.v_descale = q_descale.data_ptr(), k_descale.data_ptr(), v_descale.data_ptr()
    a.o, a.lse = out.data_ptr(), lse.data_ptr()
    a.q_strides = (ctypes.c_int64 * 3)(q8.stride(0), q8.stride(1), q8.stride(2))
    a.k_strides = (ctypes.c_int64 * 3)(k8.stride(0), k8.stride(1), k8.stride(2))
    a.vt_strides = (ctypes.c_int64 * 3)(vt8.stride(0), vt8.stride(1), vt8.stride(2))
    a.o_strides = _strides(out)
    a.causal = 1 if causal else 0
    a.q_pos_offset = FA_OFFSET_BOTTOM_RIGHT if q_pos_offset is None else int(q_pos_offset)
    a.scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    if window is not None:
        a.local = 1
        a.window_left, a.window_right = int(window[0]), int(window[1])
    check(_lib.load().fa_fwd_e4m3(ctypes.byref(a), _stream_handle(stream)), "fa_fwd_e4m3")
    return out, lse


def make_splitkv_e4m3_args(q, k8, k_descale, v8, v_descale, o, lse, *, scale=None) -> SplitkvE4m3Args:
    """Fill `fa_splitkv_e4m3_args`: q, o [b, hq, d] bf16/fp16; k8, v8 e4m3 codes (torch.uint8) [b, skv, hkv, d];
    k_descale [b, hkv, ceil(skv / 128)], v_descale [b, hkv] (fa_quantize_e4m3, V with per_head=True)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype not in _DT or q.dim() != 3 or q.stride(2) != 1:
        raise ValueError("q must be a CUDA bf16/fp16 [b, hq, d] tensor with contiguous d")
    for name, t in (("k8", k8), ("v8", v8)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.uint8 or t.dim() != 4 \
                or t.stride(3) != 1:
            raise ValueError(f"{name} must be a CUDA uint8 [b, skv, hkv, d] tensor with contiguous d")
    b, hq, d = q.shape
    skv, hkv = k8.shape[1], k8.shape[2]
    if k8.shape != (b, skv, hkv, d) or v8.shape != k8.shape or o.shape != q.shape:
        raise ValueError("inconsistent q / k8 / v8 / out shapes")
    a = SplitkvE4m3Args()
    a.dtype = _DT[q.dtype]
    a.b, a.skv, a.hq, a.hkv, a.d = b, skv, hq, hkv, d
    a.q = q.data_ptr()
    a.q_strides = (ctypes.c_int64 * 2)(q.stride(0), q.stride(1))
    a.k, a.v = k8.data_ptr(), v8.data_ptr()
    a.k_strides = (ctypes.c_int64 * 3)(k8.stride(0), k8.stride(1), k8.stride(2))
    a.v_strides = (ctypes.c_int64 * 3)(v8.stride(0), v8.stride(1), v8.stride(2))
    a.k_descale, a.v_descale = k_descale.data_ptr(), v_descale.data_ptr()
    a.o = o.data_ptr()
    a.o_strides = (ctypes.c_int64 * 2)(o.stride(0), o.stride(1))
    a.lse = lse.data_ptr()
    a.scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    return a


def fa_fwd_splitkv_e4m3(q, k8, k_descale, v8, v_descale, *, scale=None, num_splits: int = 0, workspace=None,
                        out=None, lse=None, stream=None, return_splits=False):
    """Decode one query row per (batch, head) against e4m3 keys and values; returns (O [b, hq, d], LSE [b, hq])."""
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    a = make_splitkv_e4m3_args(q, k8, k_descale, v8, v_descale, out, lse, scale=scale)
    lib = _lib.load()
    if workspace is None:
        need = int(lib.fa_splitkv_e4m3_workspace_size(ctypes.byref(a), int(num_splits)))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    used = ctypes.c_int32(0)
    check(lib.fa_fwd_splitkv_e4m3(ctypes.byref(a), int(num_splits), ctypes.c_void_p(workspace.data_ptr()),
                                  workspace.numel() * workspace.element_size(), ctypes.byref(used),
                                  _stream_handle(stream)), "fa_fwd_splitkv_e4m3")
    if return_splits:
        return out, lse, int(used.value)
    return out, lse


# What the paged cache's entry points share.  They are called once per layer and token, so their arguments are looked
# over and packed in one pass.

_NOT_ROWS = "every row tensor must be a CUDA tensor of one type (bf16 or fp16), on one device, contiguous in its last " \
    "dimension, and shaped like its counterpart"


def _enqueue(fn, args: bytes, device: int, stream, *more):
    """fn(args, *more, stream) with the tensors' device current (kernels launch on the current device)."""
    raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if device == torch.cuda.current_device():
        return fn(args, *more, raw)
    with torch.cuda.device(device):
        return fn(args, *more, raw)


def _new(stream, device, shape, dtype):
    """An uninitialised tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows3(t, device: int, dtype, n: int, h: int, d: int):
    """(pointer, row stride, head stride) of a [n, h, d] tensor; the stride of a dimension of one entry is never used
    and gets a valid value."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device or t.shape != (n, h, d):
        raise ValueError(_NOT_ROWS)
    row, head, last = t.stride()
    if last != 1:
        raise ValueError(_NOT_ROWS)
    return t.data_ptr(), row if n > 1 else d, head if h > 1 else d


def _rows4(t, device: int, dtype, shape):
    """(pointer, three strides) of a 4-D tensor, likewise."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        raise ValueError(_NOT_ROWS)
    s0, s1, s2, last = t.stride()
    if last != 1:
        raise ValueError(_NOT_ROWS)
    n0, n1, n2, d = shape
    return t.data_ptr(), s0 if n0 > 1 else d, s1 if n1 > 1 else d, s2 if n2 > 1 else d


def _pages(device: int, block_table, seqlens_k):
    """(sequences, block table, its row stride and width, lengths) of a paged cache."""
    if not isinstance(block_table, torch.Tensor) or not isinstance(seqlens_k, torch.Tensor) \
            or block_table.dtype is not torch.int32 or seqlens_k.dtype is not torch.int32 \
            or block_table.get_device() != device or seqlens_k.get_device() != device:
        raise ValueError("block_table and seqlens_k must be CUDA int32 tensors on the device of the others")
    if block_table.dim() != 2 or seqlens_k.dim() != 1:
        raise ValueError("block_table must be [b, n] and seqlens_k [b]")
    b, width = block_table.shape
    if seqlens_k.shape[0] != b:
        raise ValueError("block_table must be [b, n] and seqlens_k [b]")
    row, col = block_table.stride()
    if (col != 1 and width > 1) or (b > 1 and seqlens_k.stride(0) != 1):
        raise ValueError("block_table must be contiguous in its last dimension, seqlens_k contiguous")
    return b, block_table.data_ptr(), row, width, seqlens_k.data_ptr()


def _prefix(device: int, cu_seqlens, b: int, total: int) -> int:
    """Pointer of the prefix sums, 0 where every sequence has the same number of rows."""
    if cu_seqlens is None:
        if b == 0 or total % b:
            raise ValueError("without cu_seqlens every sequence has the same number of rows")
        return 0
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype is not torch.int32 \
            or cu_seqlens.get_device() != device or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] != b + 1 \
            or cu_seqlens.stride(0) != 1:
        raise ValueError("cu_seqlens must be a contiguous CUDA int32 vector of b + 1 prefix sums, on the device of "
                         "the others")
    return cu_seqlens.data_ptr()


def _cache4(device: int, cache, group: int, d: int, hkv):
    """(pointer, page stride, head stride, pages, page size, KV heads) of a 4-bit cache; the page size follows from
    the bytes of a page."""
    if not isinstance(cache, torch.Tensor) or cache.dtype is not torch.uint8 or cache.get_device() != device \
            or cache.dim() != 3:
        raise ValueError("cache must be a CUDA uint8 [num_pages, hkv, page bytes] tensor on the device of the others")
    if group not in (32, 64, 128) or group > d:
        raise ValueError("group must be 32, 64 or 128 and at most the head dimension")
    per_key = d + 8 * (d // group)
    pages, heads, size = cache.shape
    if hkv is not None and heads != hkv:
        raise ValueError("cache must hold the KV heads of the others")
    if size == 0 or size % (64 * per_key):
        raise ValueError(f"a page of one head holds a multiple of 64 keys of {per_key} bytes, not {size} bytes")
    sp, sh, last = cache.stride()
    if last != 1:
        raise ValueError("cache must be contiguous in its last dimension")
    return (cache.data_ptr(), sp if pages > 1 else size * heads, sh if heads > 1 else size, pages, size // per_key,
            heads)


def _append_args(device: int, k, v, block_table, seqlens_k, cu_seqlens, q, q_out, cos_sin, rotary_dim, interleaved,
                 k_cache, v_cache, cache, group) -> bytes:
    """`fa_kv_append_args` of either cache.  q, q_out: [total, hq, d]; k, v: [total, hkv, d]; cos_sin: fp32
    [max_positions, rotary_dim], cosines then sines."""
    dtype = k.dtype
    if device < 0 or dtype not in _DT or k.dim() != 3:
        raise ValueError("k must be a CUDA bf16 or fp16 [total, hkv, d] tensor")
    total, hkv, d = k.shape
    k_at, k0, k1 = _rows3(k, device, dtype, total, hkv, d)
    v_at, v0, v1 = _rows3(v, device, dtype, total, hkv, d)
    b, table, row, width, lens = _pages(device, block_table, seqlens_k)
    cu = _prefix(device, cu_seqlens, b, total)
    hq = q_at = q0 = q1 = qo_at = qo0 = qo1 = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [total, hq, d]")
        hq = q.shape[1]
        q_at, q0, q1 = _rows3(q, device, dtype, total, hq, d)
        qo_at, qo0, qo1 = _rows3(q_out, device, dtype, total, hq, d)
    elif q_out is not None:
        raise ValueError("q_out without q")
    cs_at = rot = positions = 0
    if cos_sin is not None:
        if not isinstance(cos_sin, torch.Tensor) or cos_sin.dtype is not torch.float32 \
                or cos_sin.get_device() != device or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous CUDA fp32 [max_positions, rotary_dim] tensor")
        cs_at = cos_sin.data_ptr()
        positions, rot = cos_sin.shape
        if rotary_dim is not None and rotary_dim != rot:
            raise ValueError("rotary_dim must be the width of cos_sin")
    elif rotary_dim:
        raise ValueError("a rotation needs cos_sin")
    if cache is None:
        shape = k_cache.shape
        if len(shape) != 4 or shape[2] != hkv or shape[3] != d:
            raise ValueError("k_cache and v_cache must both be [num_pages, page_size, hkv, d]")
        pages, page_size = shape[0], shape[1]
        kc, kc0, kc1, kc2 = _rows4(k_cache, device, dtype, shape)
        vc, vc0, vc1, vc2 = _rows4(v_cache, device, dtype, shape)
        return KV_APPEND.pack(_DT[dtype], b, total, hq, hkv, d, q_at, qo_at, k_at, v_at, q0, q1, qo0, qo1, k0, k1, v0,
                              v1, cu, lens, cs_at, rot, positions, 1 if interleaved else 0, pages, page_size, table,
                              row, width, kc, vc, kc0, kc1, kc2, vc0, vc1, vc2, 0, 0, 0, 0)
    c, c0, c1, pages, page_size, _ = _cache4(device, cache, group, d, hkv)
    return KV_APPEND.pack(_DT[dtype], b, total, hq, hkv, d, q_at, qo_at, k_at, v_at, q0, q1, qo0, qo1, k0, k1, v0, v1,
                          cu, lens, cs_at, rot, positions, 1 if interleaved else 0, pages, page_size, table, row, width, 0, 0,
                          0, 0, 0, 0, 0, 0, c, c0, c1, group)


def fa_kv_append(k, v, k_cache, v_cache, *, block_table, seqlens_k, cu_seqlens=None, q=None, q_out=None, cos_sin=None,
                 rotary_dim=None, interleaved: bool = False, stream=None):
    """Append new keys and values [total, hkv, d] to a paged cache [num_pages, page_size, hkv, d], rotating k (and q)
    by cos_sin at each token's position; returns the rotated q (None without q).  seqlens_k counts each sequence's
    keys after the append; cu_seqlens None: the same number of new tokens for every sequence."""
    device = k.get_device()
    if q is not None and q_out is None and device >= 0:
        q_out = _new(stream, k.device, q.shape, q.dtype)
    if not isinstance(k_cache, torch.Tensor) or not isinstance(v_cache, torch.Tensor):
        raise ValueError("k_cache and v_cache must both be [num_pages, page_size, hkv, d]")
    a = _append_args(device, k, v, block_table, seqlens_k, cu_seqlens, q, q_out, cos_sin, rotary_dim, interleaved,
                     k_cache, v_cache, None, 0)
    check(_enqueue(_lib.load().fa_kv_append, a, device, stream), "fa_kv_append")
    return q_out


def fa_kv_append_int4(k, v, cache, *, group: int, block_table, seqlens_k, cu_seqlens=None, q=None, q_out=None,
                      cos_sin=None, rotary_dim=None, interleaved: bool = False, stream=None):
    """fa_kv_append into a 4-bit cache (uint8 [num_pages, hkv, fa_kvcache_int4_page_bytes(page_size, d, group)]): one
    (scale, min) pair per token, head and group of `group` dims; returns the rotated q."""
    device = k.get_device()
    if cache is None:
        raise ValueError("a 4-bit cache is needed")
    if q is not None and q_out is None and device >= 0:
        q_out = _new(stream, k.device, q.shape, q.dtype)
    a = _append_args(device, k, v, block_table, seqlens_k, cu_seqlens, q, q_out, cos_sin, rotary_dim, interleaved,
                     None, None, cache, group)
    check(_enqueue(_lib.load().fa_kv_append_int4, a, device, stream), "fa_kv_append_int4")
    return q_out


def fa_kvcache_int4_page_bytes(page_size: int, d: int, group: int) -> int:
    """Bytes of one page of one KV head of a 4-bit cache (0: unsupported)."""
    return int(_lib.load().fa_kvcache_int4_page_bytes(int(page_size), int(d), int(group)))


def fa_kv_gather_int4(cache, *, group: int, block_table, seqlens_k, cu_seqlens=None, k_out=None, v_out=None,
                      total=None, d=None, dtype=None, stream=None):
    """The last rows of each sequence of a 4-bit cache in 16 bits: sequence s fills rows [cu_seqlens[s],
    cu_seqlens[s + 1]) of k_out and v_out [total, hkv, d] (cu_seqlens None: total / b rows each).  Without k_out
    and v_out, total, d and dtype say what to allocate.  Returns (k_out, v_out)."""
    device = cache.get_device()
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out come together")
    if device < 0 or cache.dim() != 3:
        raise ValueError("cache must be a CUDA [num_pages, hkv, page bytes] tensor")
    if k_out is None:
        if total is None or d is None or dtype is None:
            raise ValueError("total, d and dtype are needed to allocate the rows")
        shape = (int(total), cache.shape[1], int(d))
        k_out, v_out = _new(stream, cache.device, shape, dtype), _new(stream, cache.device, shape, dtype)
    dtype = k_out.dtype
    if dtype not in _DT or k_out.dim() != 3:
        raise ValueError("k_out and v_out must both be bf16 or fp16 [total, hkv, d]")
    total, hkv, d = k_out.shape
    k_at, k0, k1 = _rows3(k_out, device, dtype, total, hkv, d)
    v_at, v0, v1 = _rows3(v_out, device, dtype, total, hkv, d)
    b, table, row, width, lens = _pages(device, block_table, seqlens_k)
    cu = _prefix(device, cu_seqlens, b, total)
    c, c0, c1, pages, page_size, _ = _cache4(device, cache, group, d, hkv)
    a = KV_GATHER_INT4.pack(_DT[dtype], b, total, hkv, d, group, c, c0, c1, pages, page_size, table, row, width, lens, cu,
                            k_at, v_at, k0, k1, v0, v1)
    check(_enqueue(_lib.load().fa_kv_gather_int4, a, device, stream), "fa_kv_gather_int4")
    return k_out, v_out


def fa_fwd_kvcache_int4(q, cache, *, group: int, block_table, seqlens_k, scale=None, window_left=None,
                        softcap: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Attend the sq newest tokens of each sequence (q [b, sq, hq, d], or [b, hq, d]) to its 4-bit paged cache, each
    token to the keys up to its own; returns (O like q, LSE [b, hq, sq] or [b, hq])."""
    device, shape, dtype = q.get_device(), q.shape, q.dtype
    if device < 0 or dtype not in _DT or len(shape) not in (3, 4):
        raise ValueError("q must be a CUDA bf16 or fp16 tensor [b, sq, hq, d] or [b, hq, d]")
    if len(shape) == 4:
        b, sq, hq, d = shape
        lse_shape = (b, hq, sq)
    else:
        b, hq, d = shape
        sq, lse_shape = 1, (b, hq)
    if out is None:
        out = _new(stream, q.device, shape, dtype)
    if lse is None:
        lse = _new(stream, q.device, lse_shape, torch.float32)
    elif lse.shape != lse_shape or lse.dtype is not torch.float32 or lse.get_device() != device \
            or not lse.is_contiguous():
        raise ValueError("lse must be contiguous CUDA fp32 [b, hq, sq] (or [b, hq])")
    if len(shape) == 4:
        q_at, q0, q1, q2 = _rows4(q, device, dtype, shape)
        o_at, o0, o1, o2 = _rows4(out, device, dtype, shape)
    else:
        q_at, q0, q2 = _rows3(q, device, dtype, b, hq, d)
        o_at, o0, o2 = _rows3(out, device, dtype, b, hq, d)
        q1 = o1 = d
    seqs, table, row, width, lens = _pages(device, block_table, seqlens_k)
    if seqs != b:
        raise ValueError("block_table must be [b, n] and seqlens_k [b]")
    c, c0, c1, pages, page_size, hkv = _cache4(device, cache, group, d, None)
    a = KVCACHE_INT4.pack(_DT[dtype], b, sq, hq, hkv, d, group, q_at, q0, q1, q2, c, c0, c1, pages, page_size, table,
                          row, width, lens, o_at, o0, o1, o2, lse.data_ptr(), d ** -0.5 if scale is None else scale,
                          0 if window_left is None else 1, 0 if window_left is None else window_left, softcap)
    lib = _lib.load()
    if workspace is None:
        need = _enqueue(lambda args, _: lib.fa_kvcache_int4_workspace_size(args), a, device, stream)
        workspace = _new(stream, q.device, (max(int(need), 256),), torch.uint8)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on q's device")
    check(_enqueue(lib.fa_fwd_kvcache_int4, a, device, stream, workspace.data_ptr(),
                   workspace.numel() * workspace.element_size()), "fa_fwd_kvcache_int4")
    return out, lse


def fa_splitkv_combine(o_part, lse_part, out, lse=None, stream=None):
    """Merge fp32 partials o_part [ns, b, hq, sq, d], lse_part [ns, b, hq, sq] into out [b, sq, hq, d]."""
    ns, b, hq, sq, d = o_part.shape
    if not (o_part.is_cuda and lse_part.is_cuda and out.is_cuda):
        raise ValueError("tensors must be on the GPU")
    if o_part.dtype != torch.float32 or lse_part.dtype != torch.float32 or not o_part.is_contiguous() \
            or not lse_part.is_contiguous() or lse_part.shape != (ns, b, hq, sq):
        raise ValueError("partials must be contiguous fp32")
    if out.dtype not in _DT or out.shape != (b, sq, hq, d) or out.stride(3) != 1:
        raise ValueError("out must be [b, sq, hq, d] bf16/fp16")
    st = _strides(out)
    lp = ctypes.c_void_p(lse.data_ptr()) if lse is not None else ctypes.c_void_p(0)
    check(_lib.load().fa_splitkv_combine(ctypes.c_void_p(o_part.data_ptr()), ctypes.c_void_p(lse_part.data_ptr()),
                                         ns, b, hq, sq, d, _DT[out.dtype], ctypes.c_void_p(out.data_ptr()), st, lp,
                                         _stream_handle(stream)), "fa_splitkv_combine")
    return out, lse


def fa_sync_status(stream=None) -> int:
    """Synchronise the stream; return the status code (0 = ok, 4 = a device wait timed out)."""
    return int(_lib.load().fa_sync_status(_stream_handle(stream)))


def fa_selftest_wait_timeout(stream=None) -> None:
    check(_lib.load().fa_selftest_wait_timeout(_stream_handle(stream)), "fa_selftest_wait_timeout")


def fa_version() -> int:
    return int(_lib.load().fa_version())
