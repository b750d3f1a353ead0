"""Exact IO-aware attention for one NVIDIA GB300 (sm_103a).

Python binding of ``libfa_gb300.so``: the functions below carry the C ABI's
names (include/fa.h) and only marshal arguments.  Every step of the
attention path runs in the library's CUDA kernels; PyTorch supplies device
memory and streams.  There is no fallback: if the library cannot be built or
loaded, the first call raises.

Raw calls (``fa_forward``, ``fa_backward`` ...) take tensors or integer
device pointers, the sizes, and a stream (``None`` = PyTorch's current
stream); they return the ``fa_status`` code.  ``attention_forward`` and
``attention_backward`` allocate outputs and raise ``FaError`` on failure;
so do ``qk_norm_rope`` (and its backward), ``cache_append``,
``cache_read`` and ``tree_attention``, which also check types, shapes and
devices (``ValueError``) and run on their tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_MISALIGNED = 3
FA_ERR_WORKSPACE = 4
FA_ERR_CUDA = 5
FA_ERR_TIMEOUT = 6

FA_CACHE_BF16 = 0
FA_CACHE_E4M3 = 1
FA_CACHE_INT8 = 2

EXPORTS = (
    "fa_status_string", "fa_forward", "fa_backward_workspace_size", "fa_backward",
    "fa_backward_preprocess", "fa_backward_main", "fa_backward_dq_convert", "fa_backward_noalloc",
    "fa_blocksparse_workspace_size", "fa_blocksparse_build_lists", "fa_blocksparse_forward",
    "fa_blocksparse_backward", "fa_get_device_status", "fa_set_wait_limit_ns",
    "fa_debug_wait_timeout", "fa_debug_schedule", "fa_debug_mma_probe", "fa_forward_gqa",
    "fa_backward_gqa", "fa_debug_forward_config", "fa_forward_varlen", "fa_backward_varlen",
    "fa_forward_dropout", "fa_backward_dropout", "fa_backward_deterministic",
    "fa_qk_norm_rope", "fa_qk_norm_rope_workspace_size", "fa_qk_norm_rope_backward",
    "fa_cache_append", "fa_cache_read", "fa_tree_attention_workspace_size", "fa_tree_attention",
)

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def library_path() -> str:
    from . import build as _build
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libfa_gb300.so (building it with nvcc when absent or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        from . import build as _build
        if build_if_missing and not _build.is_fresh():
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError("libfa_gb300.so is missing: run "
                               "`python -m io_aware_exact_15_gb300.build`")
        lib = ctypes.CDLL(_build.LIB)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        U, UI = ctypes.c_ulonglong, ctypes.c_uint
        sig = {
            "fa_status_string": ([I], ctypes.c_char_p),
            "fa_forward": ([P, P, P, P, P, I, I, I, I, F, I, P], I),
            "fa_backward_workspace_size": ([I, I, I, I], Z),
            "fa_backward": ([P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, P, Z, P], I),
            "fa_backward_preprocess": ([P, P, I, I, I, I, P, Z, P], I),
            "fa_backward_main": ([P, P, P, P, P, P, P, I, I, I, I, F, I, P, Z, P], I),
            "fa_backward_dq_convert": ([P, I, I, I, I, F, P, Z, P], I),
            "fa_backward_noalloc": ([P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, P], I),
            "fa_blocksparse_workspace_size": ([I, I, I, I, I], Z),
            "fa_blocksparse_build_lists": ([P, I, I, P, Z, P], I),
            "fa_blocksparse_forward": ([P, P, P, P, P, I, I, I, I, F, I, P, I, P, Z, P], I),
            "fa_blocksparse_backward": ([P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, P, I, P, Z,
                                         P], I),
            "fa_get_device_status": ([P], I),
            "fa_set_wait_limit_ns": ([U], I),
            "fa_debug_wait_timeout": ([U, P], I),
            "fa_debug_schedule": ([I, I, P, I, P, Z, P, P, P, P, P], I),
            "fa_debug_mma_probe": ([P, P, P, I, I, P], I),
            "fa_forward_gqa": ([P, P, P, P, P, I, I, I, I, I, F, I, P], I),
            "fa_debug_forward_config": ([P, P, P, P, P, I, I, I, I, F, I, I, I, I, P], I),
            "fa_backward_gqa": ([P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, P, Z, P], I),
            "fa_forward_varlen": ([P, P, P, P, P, P, I, I, I, I, I, I, F, I, F, U, UI, P], I),
            "fa_backward_varlen": ([P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, F, U,
                                    UI, P, Z, P], I),
            "fa_forward_dropout": ([P, P, P, P, P, I, I, I, I, F, I, F, U, UI, P], I),
            "fa_backward_deterministic": ([P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, P, Z, P],
                                          I),
            "fa_backward_dropout": ([P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, F, U, UI, P, Z,
                                     P], I),
            "fa_qk_norm_rope": ([P] * 9 + [I] * 8 + [F, P, P], I),
            "fa_qk_norm_rope_workspace_size": ([I], Z),
            "fa_qk_norm_rope_backward": ([P] * 13 + [I] * 8 + [F, P, P, P, Z, P], I),
            "fa_cache_append": ([P] * 9 + [I] * 8 + [P, P], I),
            "fa_cache_read": ([P] * 9 + [I] * 8 + [P], I),
            "fa_tree_attention_workspace_size": ([I] * 5, Z),
            "fa_tree_attention": ([P] * 11 + [I] * 9 + [F, P, Z, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


# ------------------------------------------------------------------ marshalling
def _p(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _s(stream):
    if stream is None:
        import torch
        # the handle itself: a Stream object costs 3 us a call
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and torch.cuda.is_initialized():
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


# ------------------------------------------------------------------ raw C-ABI calls
def fa_status_string(status: int) -> str:
    return status_string(status)


def fa_forward(q, k, v, o, lse, B, H, N, d, scale, causal, stream=None) -> int:
    return load().fa_forward(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, N, d, float(scale),
                             int(bool(causal)), _s(stream))


def fa_forward_gqa(q, k, v, o, lse, B, H, Hkv, N, d, scale, causal, stream=None) -> int:
    return load().fa_forward_gqa(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, Hkv, N, d,
                                 float(scale), int(bool(causal)), _s(stream))


def fa_backward_gqa(q, k, v, o, dO, lse, dq, dk, dv, B, H, Hkv, N, d, scale, causal, workspace,
                    workspace_bytes, stream=None) -> int:
    return load().fa_backward_gqa(_p(q), _p(k), _p(v), _p(o), _p(dO), _p(lse), _p(dq), _p(dk),
                                  _p(dv), B, H, Hkv, N, d, float(scale), int(bool(causal)),
                                  _p(workspace), int(workspace_bytes), _s(stream))


def fa_forward_varlen(q, k, v, o, lse, cu_seqlens, B, max_seqlen, total, H, Hkv, d, scale,
                      causal, p_drop, seed, offset, stream=None) -> int:
    return load().fa_forward_varlen(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens), B,
                                    max_seqlen, total, H, Hkv, d, float(scale),
                                    int(bool(causal)), float(p_drop), int(seed), int(offset),
                                    _s(stream))


def fa_backward_varlen(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, B, max_seqlen, total, H, Hkv,
                       d, scale, causal, p_drop, seed, offset, workspace, workspace_bytes,
                       stream=None) -> int:
    return load().fa_backward_varlen(_p(q), _p(k), _p(v), _p(o), _p(dO), _p(lse), _p(dq), _p(dk),
                                     _p(dv), _p(cu_seqlens), B, max_seqlen, total, H, Hkv, d,
                                     float(scale), int(bool(causal)), float(p_drop), int(seed),
                                     int(offset), _p(workspace), int(workspace_bytes), _s(stream))


def fa_forward_dropout(q, k, v, o, lse, B, H, N, d, scale, causal, p_drop, seed, offset,
                       stream=None) -> int:
    return load().fa_forward_dropout(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, N, d,
                                     float(scale), int(bool(causal)), float(p_drop), int(seed),
                                     int(offset), _s(stream))


def fa_backward_dropout(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, p_drop, seed,
                        offset, workspace, workspace_bytes, stream=None) -> int:
    return load().fa_backward_dropout(_p(q), _p(k), _p(v), _p(o), _p(dO), _p(lse), _p(dq),
                                      _p(dk), _p(dv), B, H, N, d, float(scale), int(bool(causal)),
                                      float(p_drop), int(seed), int(offset), _p(workspace),
                                      int(workspace_bytes), _s(stream))


def fa_backward_deterministic(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal,
                              workspace, workspace_bytes, stream=None) -> int:
    return load().fa_backward_deterministic(_p(q), _p(k), _p(v), _p(o), _p(dO), _p(lse), _p(dq),
                                            _p(dk), _p(dv), B, H, N, d, float(scale),
                                            int(bool(causal)), _p(workspace),
                                            int(workspace_bytes), _s(stream))


def fa_backward_workspace_size(B, H, N, d) -> int:
    return load().fa_backward_workspace_size(B, H, N, d)


def fa_backward(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                workspace_bytes, stream=None) -> int:
    return load().fa_backward(_p(q), _p(k), _p(v), _p(o), _p(dO), _p(lse), _p(dq), _p(dk), _p(dv),
                              B, H, N, d, float(scale), int(bool(causal)), _p(workspace),
                              int(workspace_bytes), _s(stream))


def fa_backward_preprocess(o, dO, B, H, N, d, workspace, workspace_bytes, stream=None) -> int:
    return load().fa_backward_preprocess(_p(o), _p(dO), B, H, N, d, _p(workspace),
                                         int(workspace_bytes), _s(stream))


def fa_backward_main(q, k, v, dO, lse, dk, dv, B, H, N, d, scale, causal, workspace,
                     workspace_bytes, stream=None) -> int:
    return load().fa_backward_main(_p(q), _p(k), _p(v), _p(dO), _p(lse), _p(dk), _p(dv), B, H, N,
                                   d, float(scale), int(bool(causal)), _p(workspace),
                                   int(workspace_bytes), _s(stream))


def fa_backward_dq_convert(dq, B, H, N, d, scale, workspace, workspace_bytes, stream=None) -> int:
    return load().fa_backward_dq_convert(_p(dq), B, H, N, d, float(scale), _p(workspace),
                                         int(workspace_bytes), _s(stream))


def fa_backward_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal,
                        stream=None) -> int:
    """fa_backward with the library's fixed 32 MiB per-device scratch array
    instead of a caller workspace (for callers that cannot allocate)."""
    return load().fa_backward_noalloc(_p(q), _p(k), _p(v), _p(o), _p(dO), _p(lse), _p(dq), _p(dk),
                                      _p(dv), B, H, N, d, float(scale), int(bool(causal)),
                                      _s(stream))


def fa_blocksparse_workspace_size(B, H, N, d, mask_heads) -> int:
    return load().fa_blocksparse_workspace_size(B, H, N, d, mask_heads)


def fa_blocksparse_build_lists(block_mask, mask_heads, N, workspace, workspace_bytes,
                               stream=None) -> int:
    return load().fa_blocksparse_build_lists(_p(block_mask), mask_heads, N, _p(workspace),
                                             int(workspace_bytes), _s(stream))


def fa_blocksparse_forward(q, k, v, o, lse, B, H, N, d, scale, causal, block_mask, mask_heads,
                           workspace, workspace_bytes, stream=None) -> int:
    return load().fa_blocksparse_forward(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, N, d,
                                         float(scale), int(bool(causal)), _p(block_mask),
                                         mask_heads, _p(workspace), int(workspace_bytes),
                                         _s(stream))


def fa_blocksparse_backward(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, block_mask,
                            mask_heads, workspace, workspace_bytes, stream=None) -> int:
    return load().fa_blocksparse_backward(_p(q), _p(k), _p(v), _p(o), _p(dO), _p(lse), _p(dq),
                                          _p(dk), _p(dv), B, H, N, d, float(scale),
                                          int(bool(causal)), _p(block_mask), mask_heads,
                                          _p(workspace), int(workspace_bytes), _s(stream))


def _six(strides):
    """Host array of six element strides, or None."""
    if strides is None:
        return None
    if len(strides) != 6:
        raise ValueError("strides: six numbers (batch, head, row of both tensors)")
    return (ctypes.c_longlong * 6)(*strides)


def fa_qk_norm_rope(q, k, wq, wk, cos, sin, positions, q_out, k_out, B, H, Hkv, N, d, rot,
                    table_rows, interleaved, eps, strides=None, stream=None) -> int:
    return load().fa_qk_norm_rope(_p(q), _p(k), _p(wq), _p(wk), _p(cos), _p(sin), _p(positions),
                                  _p(q_out), _p(k_out), B, H, Hkv, N, d, rot, table_rows,
                                  int(bool(interleaved)), float(eps), _six(strides), _s(stream))


def fa_qk_norm_rope_workspace_size(d) -> int:
    return load().fa_qk_norm_rope_workspace_size(d)


def fa_qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions, dq, dk, dwq, dwk,
                             B, H, Hkv, N, d, rot, table_rows, interleaved, eps, strides,
                             grad_strides, workspace, workspace_bytes, stream=None) -> int:
    return load().fa_qk_norm_rope_backward(
        _p(dq_out), _p(dk_out), _p(q), _p(k), _p(wq), _p(wk), _p(cos), _p(sin), _p(positions),
        _p(dq), _p(dk), _p(dwq), _p(dwk), B, H, Hkv, N, d, rot, table_rows,
        int(bool(interleaved)), float(eps), _six(strides), _six(grad_strides), _p(workspace),
        int(workspace_bytes), _s(stream))


def fa_cache_append(k, v, page_table, start, counts, k_cache, v_cache, k_scale, v_scale, format, B,
                    Hkv, N, d, num_pages, page_size, max_pages, strides=None, stream=None) -> int:
    return load().fa_cache_append(_p(k), _p(v), _p(page_table), _p(start), _p(counts), _p(k_cache),
                                  _p(v_cache), _p(k_scale), _p(v_scale), int(format), B, Hkv, N, d,
                                  num_pages, page_size, max_pages, _six(strides), _s(stream))


def fa_cache_read(k_cache, v_cache, k_scale, v_scale, page_table, start, counts, k, v, format, B,
                  Hkv, N, d, num_pages, page_size, max_pages, stream=None) -> int:
    return load().fa_cache_read(_p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale),
                                _p(page_table), _p(start), _p(counts), _p(k), _p(v), int(format),
                                B, Hkv, N, d, num_pages, page_size, max_pages, _s(stream))


def fa_tree_attention_workspace_size(B, H, Hkv, T, d) -> int:
    return load().fa_tree_attention_workspace_size(B, H, Hkv, T, d)


def fa_tree_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, hist_lens, draft_lens,
                      tree_mask, o, lse, format, B, H, Hkv, T, d, num_pages, page_size, max_pages,
                      scale, workspace, workspace_bytes, stream=None) -> int:
    return load().fa_tree_attention(
        _p(q), _p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale), _p(page_table), _p(hist_lens),
        _p(draft_lens), _p(tree_mask), _p(o), _p(lse), int(format), B, H, Hkv, T, d, num_pages,
        page_size, max_pages, float(scale), _p(workspace), int(workspace_bytes), _s(stream))


def fa_get_device_status(stream=None) -> int:
    return load().fa_get_device_status(_s(stream))


def fa_set_wait_limit_ns(ns: int) -> int:
    return load().fa_set_wait_limit_ns(int(ns))


def fa_debug_wait_timeout(limit_ns: int, stream=None) -> int:
    return load().fa_debug_wait_timeout(int(limit_ns), _s(stream))


def fa_debug_schedule(N, causal, block_mask, mask_heads, workspace, workspace_bytes, fwd_counts,
                      bwd_counts, fwd_lists, bwd_lists, stream=None) -> int:
    return load().fa_debug_schedule(N, int(bool(causal)), _p(block_mask), mask_heads,
                                    _p(workspace), int(workspace_bytes), _p(fwd_counts),
                                    _p(bwd_counts), _p(fwd_lists), _p(bwd_lists), _s(stream))


def fa_debug_forward_config(q, k, v, o, lse, B, H, N, d, scale, causal, rows_per_cta,
                            key_tile, kv_stages, stream=None) -> int:
    return load().fa_debug_forward_config(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, N, d,
                                          float(scale), int(bool(causal)), int(rows_per_cta),
                                          int(key_tile), int(kv_stages), _s(stream))


def fa_debug_mma_probe(a, b, c, mode, n, stream=None) -> int:
    return load().fa_debug_mma_probe(_p(a), _p(b), _p(c), int(mode), int(n), _s(stream))


# ------------------------------------------------------------------ allocating wrappers
def _check(status, what):
    if status != FA_OK:
        raise FaError(status, what)


def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    return tuple(int(x) for x in q.shape)


def _varlen_shape(q, k, cu_seqlens, max_seqlen):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("variable-length batches take [H, total, d] tensors")
    H, T, d = (int(x) for x in q.shape)
    B = int(cu_seqlens.numel()) - 1
    if B < 1:
        raise ValueError("cu_seqlens needs B + 1 >= 2 entries")
    if max_seqlen is None:  # one host read of the offsets
        cu = cu_seqlens.cpu()
        max_seqlen = int((cu[1:] - cu[:-1]).max()) if T > 0 else 0
    return B, H, int(k.shape[0]), T, d, int(max_seqlen)


def attention_forward(q, k, v, scale=None, causal=False, block_mask=None, workspace=None,
                      stream=None, cu_seqlens=None, max_seqlen=None, dropout_p=0.0, seed=0,
                      offset=0):
    """(o, lse) for bf16 CUDA tensors q [B, H, N, d] and k, v [B, Hkv, N, d]
    (Hkv = H, or a divisor of H for grouped heads).  With cu_seqlens (int32
    CUDA tensor [B+1]) the batch is packed: q [H, total, d], k, v
    [Hkv, total, d], lse [H, total].  dropout_p > 0: dropout on P with the
    Philox keep rule of (seed, offset); the backward must get the same."""
    import torch
    if cu_seqlens is not None:
        if block_mask is not None:
            raise ValueError("block masks apply to equal-length batches only")
        B, H, Hkv, T, d, ms = _varlen_shape(q, k, cu_seqlens, max_seqlen)
        scale = (1.0 / d ** 0.5) if scale is None else scale
        o = torch.empty_like(q)
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
        _check(fa_forward_varlen(q, k, v, o, lse, cu_seqlens, B, ms, T, H, Hkv, d, scale, causal,
                                 dropout_p, seed, offset, stream), "fa_forward_varlen")
        return o, lse
    B, H, N, d = _shape(q)
    Hkv = int(k.shape[1])
    scale = (1.0 / d ** 0.5) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if dropout_p:
        if block_mask is not None or Hkv != H:
            raise ValueError("dropout applies to dense Hkv = H or variable-length batches")
        _check(fa_forward_dropout(q, k, v, o, lse, B, H, N, d, scale, causal, dropout_p, seed,
                                  offset, stream), "fa_forward_dropout")
    elif block_mask is None:
        if Hkv == H:
            _check(fa_forward(q, k, v, o, lse, B, H, N, d, scale, causal, stream), "fa_forward")
        else:
            _check(fa_forward_gqa(q, k, v, o, lse, B, H, Hkv, N, d, scale, causal, stream),
                   "fa_forward_gqa")
    else:
        if Hkv != H:
            raise ValueError("block masks apply to Hkv = H only")
        mh = int(block_mask.shape[0])
        nbytes = fa_blocksparse_workspace_size(B, H, N, d, mh)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        _check(fa_blocksparse_forward(q, k, v, o, lse, B, H, N, d, scale, causal, block_mask, mh,
                                      workspace, workspace.numel(), stream),
               "fa_blocksparse_forward")
    return o, lse


def attention_backward(q, k, v, o, dO, lse, scale=None, causal=False, block_mask=None,
                       workspace=None, stream=None, cu_seqlens=None, max_seqlen=None,
                       dropout_p=0.0, seed=0, offset=0):
    """(dq, dk, dv) of sum(O * dO); shapes and options as attention_forward."""
    import torch
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if cu_seqlens is not None:
        if block_mask is not None:
            raise ValueError("block masks apply to equal-length batches only")
        B, H, Hkv, T, d, ms = _varlen_shape(q, k, cu_seqlens, max_seqlen)
        scale = (1.0 / d ** 0.5) if scale is None else scale
        nbytes = fa_backward_workspace_size(1, H, max(T, 1), d)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        _check(fa_backward_varlen(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, B, ms, T, H, Hkv, d,
                                  scale, causal, dropout_p, seed, offset, workspace,
                                  workspace.numel(), stream), "fa_backward_varlen")
        return dq, dk, dv
    B, H, N, d = _shape(q)
    Hkv = int(k.shape[1])
    scale = (1.0 / d ** 0.5) if scale is None else scale
    if dropout_p:
        if block_mask is not None or Hkv != H:
            raise ValueError("dropout applies to dense Hkv = H or variable-length batches")
        nbytes = fa_backward_workspace_size(B, H, N, d)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        _check(fa_backward_dropout(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal,
                                   dropout_p, seed, offset, workspace, workspace.numel(), stream),
               "fa_backward_dropout")
    elif block_mask is None:
        nbytes = fa_backward_workspace_size(B, H, N, d)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        if Hkv == H:
            _check(fa_backward(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal,
                               workspace, workspace.numel(), stream), "fa_backward")
        else:
            _check(fa_backward_gqa(q, k, v, o, dO, lse, dq, dk, dv, B, H, Hkv, N, d, scale, causal,
                                   workspace, workspace.numel(), stream), "fa_backward_gqa")
    else:
        if Hkv != H:
            raise ValueError("block masks apply to Hkv = H only")
        mh = int(block_mask.shape[0])
        nbytes = fa_blocksparse_workspace_size(B, H, N, d, mh)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        _check(fa_blocksparse_backward(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal,
                                       block_mask, mh, workspace, workspace.numel(), stream),
               "fa_blocksparse_backward")
    return dq, dk, dv


# ------------------------------------------------------------------ Q/K preparation and serving
def _want(name, t, shape, dtypes, like, contiguous=True):
    """Refuses a tensor of another type, shape or device than the call needs."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.device != like.device or not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a CUDA tensor on {like.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _bytes(workspace, like):
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be contiguous on {like.device}")
    return workspace.numel() * workspace.element_size()


@contextlib.contextmanager
def _launch_on(t, stream):
    """Makes t's device current, and `stream` too where one is given, so that
    what the wrapper allocates belongs to the stream its kernels run on."""
    import torch
    with torch.cuda.device(t.device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=t.device)
        if stream.device != t.device:
            raise ValueError(f"stream on {stream.device}, tensors on {t.device}")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def _heads(q, k, names=("q", "k")):
    import torch
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"{names[0]}, {names[1]}: expected [B, heads, N, d]")
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    for name, t, h in ((names[0], q, H), (names[1], k, Hkv)):
        _want(name, t, (B, h, N, d), (torch.bfloat16,), q, contiguous=False)
        if t.stride(3) != 1 and d > 1:
            raise ValueError(f"{name}: the d elements of a row must be contiguous")
    return B, H, Hkv, N, d


def _rope_args(q, k, wq, wk, cos, sin, positions):
    import torch
    B, H, Hkv, N, d = _heads(q, k)
    f32 = (torch.float32,)
    if cos.dim() != 2:
        raise ValueError("cos, sin: expected [table_rows, rot / 2]")
    _want("wq", wq, (d,), f32, q)
    _want("wk", wk, (d,), f32, q)
    _want("cos", cos, cos.shape, f32, q)
    _want("sin", sin, cos.shape, f32, q)
    if positions is not None:
        _want("positions", positions, (B, N), (torch.int32,), q)
    return B, H, Hkv, N, d, 2 * cos.shape[1], cos.shape[0]


def qk_norm_rope(q, k, wq, wk, cos, sin, positions=None, eps=1e-6, interleaved=False, stream=None):
    """(q_out, k_out), contiguous bf16 [B, H, N, d] and [B, Hkv, N, d]: the
    rows of q and k normed per head, weighted by wq, wk (fp32 [d]) and turned
    by the rows `positions` (int32 [B, N]; None: 0 .. N-1) of cos, sin (fp32
    [table_rows, rot / 2]).  q and k may be strided views, for instance
    ``qkv[:, :, :H].transpose(1, 2)`` of a packed [B, N, H + 2 Hkv, d]
    projection."""
    import torch
    sizes = _rope_args(q, k, wq, wk, cos, sin, positions)
    B, H, Hkv, N, d = sizes[:5]
    with _launch_on(q, stream) as s:
        q_out = torch.empty((B, H, N, d), dtype=q.dtype, device=q.device)
        k_out = torch.empty((B, Hkv, N, d), dtype=q.dtype, device=q.device)
        _check(fa_qk_norm_rope(q, k, wq, wk, cos, sin, positions, q_out, k_out, *sizes,
                               interleaved, eps, q.stride()[:3] + k.stride()[:3], s),
               "fa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions=None, eps=1e-6,
                          interleaved=False, dq=None, dk=None, workspace=None, stream=None):
    """(dq, dk, dwq, dwk) of qk_norm_rope; dq_out, dk_out contiguous.  dq, dk
    may be given (views of a packed gradient, say); otherwise they are
    contiguous [B, H, N, d] and [B, Hkv, N, d]."""
    import torch
    sizes = _rope_args(q, k, wq, wk, cos, sin, positions)
    B, H, Hkv, N, d = sizes[:5]
    bf16 = (torch.bfloat16,)
    _want("dq_out", dq_out, (B, H, N, d), bf16, q)
    _want("dk_out", dk_out, (B, Hkv, N, d), bf16, q)
    for name, t, h in (("dq", dq, H), ("dk", dk, Hkv)):
        if t is not None:
            _want(name, t, (B, h, N, d), bf16, q, contiguous=False)
            if t.stride(3) != 1:
                raise ValueError(f"{name}: the d elements of a row must be contiguous")
    with _launch_on(q, stream) as s:
        new = lambda *shape, dtype=q.dtype: torch.empty(shape, dtype=dtype, device=q.device)
        dq = new(B, H, N, d) if dq is None else dq
        dk = new(B, Hkv, N, d) if dk is None else dk
        dwq, dwk = new(d, dtype=torch.float32), new(d, dtype=torch.float32)
        if workspace is None:
            workspace = new(fa_qk_norm_rope_workspace_size(d), dtype=torch.uint8)
        _check(fa_qk_norm_rope_backward(
            dq_out, dk_out, q, k, wq, wk, cos, sin, positions, dq, dk, dwq, dwk, *sizes,
            interleaved, eps, q.stride()[:3] + k.stride()[:3], dq.stride()[:3] + dk.stride()[:3],
            workspace, _bytes(workspace, q), s),
            "fa_qk_norm_rope_backward")
    return dq, dk, dwq, dwk


def _cache_args(k_cache, v_cache, k_scale, v_scale, page_table, B):
    """(format, (num_pages, page_size, max_pages), Hkv, d) of a paged cache;
    the format follows from the caches' type."""
    import torch
    if k_cache.dim() != 4:
        raise ValueError("caches: expected [num_pages, Hkv, page_size, d]")
    formats = {torch.bfloat16: FA_CACHE_BF16, torch.float8_e4m3fn: FA_CACHE_E4M3,
               torch.int8: FA_CACHE_INT8}
    if k_cache.dtype not in formats:
        raise ValueError(f"caches: {k_cache.dtype}, expected bfloat16, float8_e4m3fn or int8")
    num_pages, Hkv, page_size, d = k_cache.shape
    _want("k_cache", k_cache, k_cache.shape, (k_cache.dtype,), k_cache)
    _want("v_cache", v_cache, k_cache.shape, (k_cache.dtype,), k_cache)
    fmt = formats[k_cache.dtype]
    if fmt != FA_CACHE_BF16:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        _want("k_scale", k_scale, k_cache.shape[:3], (torch.uint8,), k_cache)
        _want("v_scale", v_scale, k_cache.shape[:3], (torch.uint8,), k_cache)
    if page_table.dim() != 2:
        raise ValueError("page_table: expected [B, max_pages]")
    _want("page_table", page_table, (B, page_table.shape[1]), (torch.int32,), k_cache)
    return fmt, (num_pages, page_size, page_table.shape[1]), Hkv, d


def _lens(name, t, B, like):
    import torch
    if t is not None:
        _want(name, t, (B,), (torch.int32,), like)


def cache_append(k, v, k_cache, v_cache, page_table, start, counts=None, k_scale=None, v_scale=None,
                 stream=None):
    """Writes k, v (bf16 [B, Hkv, N, d], any strides) into the paged cache:
    token n of sequence b, n < counts[b] (None: N), at position start[b] + n.
    The caches' type is the format: bfloat16, float8_e4m3fn or int8, the last
    two with scale bytes uint8 [num_pages, Hkv, page_size]."""
    B, Hk, Hv, N, d = _heads(k, v, ("k", "v"))
    fmt, pages, Hkv, dc = _cache_args(k_cache, v_cache, k_scale, v_scale, page_table, B)
    if (Hk, Hv, d) != (Hkv, Hkv, dc) or k.device != k_cache.device:
        raise ValueError("k, v and the caches differ in heads, head size or device")
    _lens("start", start, B, k)
    _lens("counts", counts, B, k)
    with _launch_on(k, stream) as s:
        _check(fa_cache_append(k, v, page_table, start, counts, k_cache, v_cache, k_scale, v_scale,
                               fmt, B, Hkv, N, d, *pages, k.stride()[:3] + v.stride()[:3], s),
               "fa_cache_append")


def cache_read(k_cache, v_cache, page_table, start, N, counts=None, k_scale=None, v_scale=None,
               stream=None):
    """(k, v), bf16 [B, Hkv, N, d]: positions start[b] .. start[b] + counts[b]
    - 1 (counts None: N of them) of each sequence; rows behind are zeros."""
    import torch
    B = int(page_table.shape[0])
    fmt, pages, Hkv, d = _cache_args(k_cache, v_cache, k_scale, v_scale, page_table, B)
    _lens("start", start, B, k_cache)
    _lens("counts", counts, B, k_cache)
    with _launch_on(k_cache, stream) as s:
        make = torch.empty if counts is None else torch.zeros
        k = make((B, Hkv, N, d), dtype=torch.bfloat16, device=k_cache.device)
        v = make((B, Hkv, N, d), dtype=torch.bfloat16, device=k_cache.device)
        _check(fa_cache_read(k_cache, v_cache, k_scale, v_scale, page_table, start, counts, k, v,
                             fmt, B, Hkv, N, d, *pages, s), "fa_cache_read")
    return k, v


def tree_attention(q, k_cache, v_cache, page_table, hist_lens, draft_lens=None, tree_mask=None,
                   scale=None, k_scale=None, v_scale=None, workspace=None, stream=None):
    """(o, lse) of drafted tokens q [B, H, T, d] over the paged cache, their
    own keys and values appended behind the hist_lens[b] accepted tokens.
    tree_mask: int32 [B, T, ceil(T / 32)], bit j of row i set when draft i
    sees draft j; None: a chain (T = 1: a plain decode step).  draft_lens
    (int32 [B], None: T): rows behind get o = 0, lse = -inf."""
    import torch
    if q.dim() != 4:
        raise ValueError("expected q [B, H, T, d]")
    B, H, T, d = q.shape
    _want("q", q, q.shape, (torch.bfloat16,), q)
    fmt, pages, Hkv, dc = _cache_args(k_cache, v_cache, k_scale, v_scale, page_table, B)
    if d != dc or q.device != k_cache.device:
        raise ValueError("q and the caches differ in head size or device")
    _lens("hist_lens", hist_lens, B, q)
    _lens("draft_lens", draft_lens, B, q)
    if tree_mask is not None:
        _want("tree_mask", tree_mask, (B, T, (T + 31) // 32), (torch.int32,), q)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    with _launch_on(q, stream) as s:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = torch.empty(fa_tree_attention_workspace_size(B, H, Hkv, T, d),
                                    dtype=torch.uint8, device=q.device)
        _check(fa_tree_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, hist_lens,
                                 draft_lens, tree_mask, o, lse, fmt, B, H, Hkv, T, d, *pages,
                                 scale, workspace, _bytes(workspace, q), s), "fa_tree_attention")
    return o, lse
