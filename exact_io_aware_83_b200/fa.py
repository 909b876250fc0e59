"""Python binding of ``libfa_sm100.so`` (declared in ``include/fa.h``).

Argument marshalling only: every step of the forward and backward pass runs in the
library's CUDA kernels.  PyTorch provides device memory and the current stream.  There
is no fallback: if the library cannot be loaded, or a call returns an error status,
:class:`FAError` is raised.

Entry points mirror the C ABI names:

* :func:`fa_fwd` / :func:`fa_bwd` - pointer-level calls (device pointers as ints);
* :func:`fa_fwd_window` / :func:`fa_bwd_window` - the same for local attention (key j
  visible to query i iff i - left <= j <= i + right, -1 = unlimited);
* :func:`fa_fwd_varlen` / :func:`fa_bwd_varlen` - packed variable-length sequences
  ([total, H, d] rows, [B+1] offsets; query and key lengths may differ, the band being
  aligned to the end of each sequence);
* :func:`fa_fwd_dropout` / :func:`fa_bwd_dropout` - attention dropout with a
  Philox4x32-10 keep mask regenerated in the backward;
* :func:`fa_fwd_blocksparse` / :func:`fa_bwd_blocksparse` - block-sparse attention over a
  per-head 0/1 mask of 128 x 128 blocks (with or without the causal mask);
* :func:`fa_decode` / :func:`fa_merge` - a few new query rows against a long key/value
  cache, split over the cache, and the merge of partial results;
* :func:`fwd` / :func:`bwd` / :func:`fwd_varlen` / :func:`bwd_varlen` / :func:`decode` /
  :func:`merge` - tensor conveniences that allocate outputs with torch
  (``window=(left, right)`` selects local attention, ``dropout_p`` / ``seed`` dropout,
  ``block_mask`` block-sparse attention; ``softcap``, ``alibi_slopes``, ``key_range`` changed
  scores);
* :func:`fa_fwd_score` / :func:`fa_bwd_score` / :func:`fa_decode_score` - attention with
  changed scores: a tanh cap, a bias that falls with the distance, a key range per query row
  (:func:`document_ranges`, :func:`prefix_ranges`);
* :func:`kv4_alloc` / :func:`kv4_write` / :func:`kv4_read` / :func:`decode_kv4` - a key/value
  cache held in 4 bits: allocated, written, read back, attended to;
* :func:`fa_bwd_workspace_bytes`, :func:`fa_device_status`, :func:`fa_status_string`.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import functools
import math
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa_sm100.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_GQA = 3
FA_ERR_ALIGN = 4
FA_ERR_WORKSPACE = 5
FA_ERR_CUDA = 6
FA_ERR_DEVICE_TIMEOUT = 7
FA_ERR_SCRATCH_LIMIT = 8
FA_ERR_SEQLENS = 9
FA_NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None
_lock = threading.Lock()


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: status {code} ({fa_status_string(code)})")


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load the library (building it with nvcc first if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            if not build_if_missing:
                raise FAError(FA_ERR_CUDA, f"library missing: {LIB_PATH}")
            from . import build as _build
            _build.build()
        lib = ctypes.CDLL(LIB_PATH)
        vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_fwd.restype = ci
        lib.fa_bwd_workspace_bytes.argtypes = [ci, ci, ci, ci, ci]
        lib.fa_bwd_workspace_bytes.restype = sz
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                               ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_bwd.restype = ci
        lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_fwd_window.restype = ci
        lib.fa_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                      ci, ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_bwd_window.restype = ci
        lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci,
                                      ci, ci, ci, cf, vp]
        lib.fa_fwd_varlen.restype = ci
        lib.fa_bwd_varlen_workspace_bytes.argtypes = [ci, ci, ci]
        lib.fa_bwd_varlen_workspace_bytes.restype = sz
        lib.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp,
                                      ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_bwd_varlen.restype = ci
        u64 = ctypes.c_ulonglong
        lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, u64, cf, vp]
        lib.fa_fwd_dropout.restype = ci
        lib.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                       ci, ci, ci, ci, ci, ci, cf, u64, cf, vp]
        lib.fa_bwd_dropout.restype = ci
        lib.fa_fwd_blocksparse.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_fwd_blocksparse.restype = ci
        lib.fa_bwd_blocksparse.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                           ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_bwd_blocksparse.restype = ci
        lib.fa_decode_num_splits.argtypes = [ci, ci, ci, ci, ci, ci]
        lib.fa_decode_num_splits.restype = ci
        lib.fa_decode_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci, ci]
        lib.fa_decode_workspace_bytes.restype = sz
        lib.fa_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, ci, ci, ci, ci, ci, ci, ci, ci,
                                  cf, vp]
        lib.fa_decode.restype = ci
        lib.fa_fwd_score.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, cf, vp]
        lib.fa_fwd_score.restype = ci
        lib.fa_bwd_score_workspace_bytes.argtypes = [ci, ci, ci, ci, ci]
        lib.fa_bwd_score_workspace_bytes.restype = sz
        lib.fa_bwd_score.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, ci, ci, ci,
                                     ci, ci, ci, cf, cf, vp]
        lib.fa_bwd_score.restype = ci
        lib.fa_decode_score.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, sz, ci, ci, ci, ci, ci, ci,
                                        ci, ci, cf, cf, vp]
        lib.fa_decode_score.restype = ci
        lib.fa_decode_score_num_splits.argtypes = [ci, ci, ci, ci, ci, ci]
        lib.fa_decode_score_num_splits.restype = ci
        lib.fa_decode_score_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci, ci]
        lib.fa_decode_score_workspace_bytes.restype = sz
        lib.fa_kv4_write.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, vp]
        lib.fa_kv4_write.restype = ci
        lib.fa_kv4_read.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, vp]
        lib.fa_kv4_read.restype = ci
        lib.fa_decode_kv4.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, ci, ci, ci, ci,
                                      ci, ci, ci, ci, cf, cf, vp]
        lib.fa_decode_kv4.restype = ci
        lib.fa_decode_kv4_num_splits.argtypes = [ci, ci, ci, ci, ci, ci]
        lib.fa_decode_kv4_num_splits.restype = ci
        lib.fa_decode_kv4_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci, ci]
        lib.fa_decode_kv4_workspace_bytes.restype = sz
        lib.fa_merge.argtypes = [vp, vp, vp, vp, ci, ci, ci, vp]
        lib.fa_merge.restype = ci
        lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                       ci, ci, ci, ci, ci, ci, cf, vp]
        lib.fa_bwd_noalloc.restype = ci
        lib.fa_device_status.argtypes = [vp]
        lib.fa_device_status.restype = ci
        lib.fa_status_string.argtypes = [ci]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_version.argtypes = []
        lib.fa_version.restype = ci
        lib.fa_watchdog_selftest.argtypes = [ci, vp]
        lib.fa_watchdog_selftest.restype = ci
        lib.fa_kernel_timing.argtypes = [ci]
        lib.fa_kernel_timing.restype = ci
        lib.fa_kernel_time_ms.argtypes = [ci, ctypes.POINTER(ctypes.c_float),
                                          ctypes.POINTER(ctypes.c_int)]
        lib.fa_kernel_time_ms.restype = ci
        lib.fa_set_fwd_scheduler.argtypes = [ci]
        lib.fa_set_fwd_scheduler.restype = ci
        lib.fa_get_fwd_scheduler.argtypes = []
        lib.fa_get_fwd_scheduler.restype = ci
        _lib = lib
        return lib


def fa_status_string(code: int) -> str:
    return load().fa_status_string(int(code)).decode()


def _check(rc: int, where: str) -> None:
    if rc != FA_OK:
        raise FAError(rc, where)


# ----------------------------------------------------------------------------- C ABI

def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, stream) -> None:
    _check(load().fa_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, int(causal), float(scale), stream),
           "fa_fwd")


def fa_fwd_window(q, k, v, o, lse, B, Hq, Hkv, N, d, window_left, window_right, scale,
                  stream) -> None:
    _check(load().fa_fwd_window(q, k, v, o, lse, B, Hq, Hkv, N, d, int(window_left),
                                int(window_right), float(scale), stream), "fa_fwd_window")


def fa_bwd_workspace_bytes(B, Hq, Hkv, N, d) -> int:
    return int(load().fa_bwd_workspace_bytes(B, Hq, Hkv, N, d))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, N, d,
           causal, scale, stream) -> None:
    _check(load().fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes,
                         B, Hq, Hkv, N, d, int(causal), float(scale), stream), "fa_bwd")


def fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, N,
                  d, window_left, window_right, scale, stream) -> None:
    _check(load().fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes,
                                B, Hq, Hkv, N, d, int(window_left), int(window_right),
                                float(scale), stream), "fa_bwd_window")


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale,
                   stream) -> None:
    """fa_bwd for callers that cannot allocate device memory: the scratch is a static
    64 MiB device buffer inside the library (see include/fa.h for the size limit and the
    rule that calls overlapping on the GPU race on that buffer)."""
    _check(load().fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, N, d,
                                 int(causal), float(scale), stream), "fa_bwd_noalloc")


def fa_fwd_varlen(q, k, v, o, lse, cu_q, cu_k, B, Hq, Hkv, total_q, total_k, max_q, max_k, d,
                  window_left, window_right, scale, stream) -> None:
    _check(load().fa_fwd_varlen(q, k, v, o, lse, cu_q, cu_k, B, Hq, Hkv, total_q, total_k, max_q,
                                max_k, d, int(window_left), int(window_right), float(scale),
                                stream), "fa_fwd_varlen")


def fa_bwd_varlen_workspace_bytes(Hq, total_q, d) -> int:
    return int(load().fa_bwd_varlen_workspace_bytes(Hq, total_q, d))


def fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, cu_q, cu_k, B,
                  Hq, Hkv, total_q, total_k, max_q, max_k, d, window_left, window_right, scale,
                  stream) -> None:
    _check(load().fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes,
                                cu_q, cu_k, B, Hq, Hkv, total_q, total_k, max_q, max_k, d,
                                int(window_left), int(window_right), float(scale), stream),
           "fa_bwd_varlen")


def fa_fwd_dropout(q, k, v, o, lse, B, Hq, Hkv, N, d, causal, dropout_p, seed, scale,
                   stream) -> None:
    _check(load().fa_fwd_dropout(q, k, v, o, lse, B, Hq, Hkv, N, d, int(causal), float(dropout_p),
                                 int(seed) & 0xFFFFFFFFFFFFFFFF, float(scale), stream),
           "fa_fwd_dropout")


def fa_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, N,
                   d, causal, dropout_p, seed, scale, stream) -> None:
    _check(load().fa_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes,
                                 B, Hq, Hkv, N, d, int(causal), float(dropout_p),
                                 int(seed) & 0xFFFFFFFFFFFFFFFF, float(scale), stream),
           "fa_bwd_dropout")


def fa_fwd_blocksparse(q, k, v, o, lse, block_mask, B, Hq, Hkv, N, d, causal, scale,
                       stream) -> None:
    _check(load().fa_fwd_blocksparse(q, k, v, o, lse, block_mask, B, Hq, Hkv, N, d, int(causal),
                                     float(scale), stream),
           "fa_fwd_blocksparse")


def fa_bwd_blocksparse(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, block_mask,
                       B, Hq, Hkv, N, d, causal, scale, stream) -> None:
    _check(load().fa_bwd_blocksparse(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes,
                                     block_mask, B, Hq, Hkv, N, d, int(causal), float(scale),
                                     stream),
           "fa_bwd_blocksparse")


def fa_decode_num_splits(B, Hq, Hkv, Nq, Nk, d) -> int:
    return int(load().fa_decode_num_splits(B, Hq, Hkv, Nq, Nk, d))


def fa_decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits) -> int:
    return int(load().fa_decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits))


def fa_decode(q, k, v, o, lse, seqlens_k, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nk, d,
              causal, num_splits, scale, stream) -> None:
    _check(load().fa_decode(q, k, v, o, lse, seqlens_k, workspace, workspace_bytes, B, Hq, Hkv,
                            Nq, Nk, d, int(causal), int(num_splits), float(scale), stream),
           "fa_decode")


def _cap(softcap) -> float:
    """A cap as C takes it: positive ones stay positive and finite in fp32."""
    c = float(softcap)
    return min(max(c, 2.0 ** -126), 2.0 ** 126) if 0.0 < c < math.inf else c


def fa_fwd_score(q, k, v, o, lse, alibi_slopes, key_range, B, Hq, Hkv, N, d, causal, softcap, scale,
                 stream) -> None:
    _check(load().fa_fwd_score(q, k, v, o, lse, alibi_slopes, key_range, B, Hq, Hkv, N, d,
                               int(causal), _cap(softcap), float(scale), stream), "fa_fwd_score")


def fa_bwd_score_workspace_bytes(B, Hq, Hkv, N, d) -> int:
    return int(load().fa_bwd_score_workspace_bytes(B, Hq, Hkv, N, d))


def fa_bwd_score(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, alibi_slopes,
                 key_range, B, Hq, Hkv, N, d, causal, softcap, scale, stream) -> None:
    _check(load().fa_bwd_score(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes,
                               alibi_slopes, key_range, B, Hq, Hkv, N, d, int(causal),
                               _cap(softcap), float(scale), stream), "fa_bwd_score")


def fa_decode_score_num_splits(B, Hq, Hkv, Nq, Nk, d) -> int:
    return int(load().fa_decode_score_num_splits(B, Hq, Hkv, Nq, Nk, d))


def fa_decode_score_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits) -> int:
    return int(load().fa_decode_score_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits))


def fa_decode_score(q, k, v, o, lse, seqlens_k, alibi_slopes, workspace, workspace_bytes, B, Hq,
                    Hkv, Nq, Nk, d, causal, num_splits, softcap, scale, stream) -> None:
    _check(load().fa_decode_score(q, k, v, o, lse, seqlens_k, alibi_slopes, workspace,
                                  workspace_bytes, B, Hq, Hkv, Nq, Nk, d, int(causal),
                                  int(num_splits), _cap(softcap), float(scale), stream),
           "fa_decode_score")


def fa_kv4_write(k, v, k_codes, k_params, v_codes, v_params, start, counts, B, Hkv, n, cap, d,
                 stream) -> None:
    _check(load().fa_kv4_write(k, v, k_codes, k_params, v_codes, v_params, start, counts, B, Hkv,
                               n, cap, d, stream), "fa_kv4_write")


def fa_kv4_read(k_codes, k_params, v_codes, v_params, k, v, start, B, Hkv, n, cap, d,
                stream) -> None:
    _check(load().fa_kv4_read(k_codes, k_params, v_codes, v_params, k, v, start, B, Hkv, n, cap,
                              d, stream), "fa_kv4_read")


def fa_decode_kv4_num_splits(B, Hq, Hkv, Nq, cap, d) -> int:
    return int(load().fa_decode_kv4_num_splits(B, Hq, Hkv, Nq, cap, d))


def fa_decode_kv4_workspace_bytes(B, Hq, Hkv, Nq, cap, d, num_splits) -> int:
    return int(load().fa_decode_kv4_workspace_bytes(B, Hq, Hkv, Nq, cap, d, num_splits))


def fa_decode_kv4(q, k_codes, k_params, v_codes, v_params, o, lse, seqlens_k, alibi_slopes,
                  workspace, workspace_bytes, B, Hq, Hkv, Nq, cap, d, causal, num_splits, softcap,
                  scale, stream) -> None:
    _check(load().fa_decode_kv4(q, k_codes, k_params, v_codes, v_params, o, lse, seqlens_k,
                                alibi_slopes, workspace, workspace_bytes, B, Hq, Hkv, Nq, cap, d,
                                int(causal), int(num_splits), _cap(softcap), float(scale),
                                stream), "fa_decode_kv4")


def fa_merge(o_parts, lse_parts, o, lse, num_parts, rows, d, stream) -> None:
    _check(load().fa_merge(o_parts, lse_parts, o, lse, int(num_parts), int(rows), int(d),
                           stream), "fa_merge")


def fa_device_status(stream=None) -> int:
    return int(load().fa_device_status(stream))


def fa_watchdog_selftest(limit_us: int, stream=None) -> None:
    _check(load().fa_watchdog_selftest(int(limit_us), stream), "fa_watchdog_selftest")


def fa_kernel_timing(enable: bool) -> None:
    _check(load().fa_kernel_timing(1 if enable else 0), "fa_kernel_timing")


def fa_set_fwd_scheduler(persistent: bool) -> bool:
    """Choose the dense forward's tile scheduler (True: persistent CTAs with dynamic unit
    assignment, False: one CTA per unit); returns the previous choice."""
    prev = load().fa_set_fwd_scheduler(1 if persistent else 0)
    if prev < 0:
        _check(prev, "fa_set_fwd_scheduler")
    return bool(prev)


def fa_get_fwd_scheduler() -> bool:
    """True when the dense forward uses the persistent scheduler."""
    return bool(load().fa_get_fwd_scheduler())


def fa_kernel_time_ms(which: int):
    """(summed device ms, launches) of the forward (0) or backward main (1) kernel."""
    ms = ctypes.c_float()
    n = ctypes.c_int()
    _check(load().fa_kernel_time_ms(int(which), ctypes.byref(ms), ctypes.byref(n)),
           "fa_kernel_time_ms")
    return float(ms.value), int(n.value)


# ----------------------------------------------------------------------------- tensors

def _stream_handle(t):
    """cudaStream_t of the current stream of t's device."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # 0.1 us against 2.4 us
    return raw(t.get_device()) if raw else torch.cuda.current_stream(t.device).cuda_stream


_HERE = contextlib.nullcontext()


def _on(t):
    """Context in which t's device is the current one."""
    import torch
    get = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device  # 0.1 us against 0.6 us
    return _HERE if get() == t.get_device() else torch.cuda.device(t.device)


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, Hq, N, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if (Bk, Nk, dk) != (B, N, d):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)}")
    return B, Hq, Hkv, N, d


def _need(t, name):
    import torch
    if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def _window(causal, window):
    if window is None:
        return None
    if causal:
        raise ValueError("give either causal=True or window=(left, right), not both")
    left, right = (int(w) for w in window)
    return left, right


def _block_mask(block_mask, B, Hq, N, win, dropout_p):
    import torch
    if block_mask is None:
        return None
    nb = (N + 127) // 128
    if block_mask.dtype == torch.bool:
        block_mask = block_mask.view(torch.uint8)  # one byte, 0 or 1, per block
    if (not block_mask.is_cuda or block_mask.dtype != torch.uint8 or not block_mask.is_contiguous()
            or tuple(block_mask.shape) != (B, Hq, nb, nb)):
        raise ValueError(f"block_mask must be a contiguous uint8 CUDA tensor [{B}, {Hq}, {nb}, {nb}]")
    if win is not None or dropout_p:
        raise ValueError("block_mask combines with causal only (no window, no dropout)")
    return block_mask


def _int32_vector(t, name, B, device):
    """Device pointer of an int32 [B] tensor (None stays None)."""
    import torch
    if t is None:
        return None
    if (not t.is_cuda or t.dtype is not torch.int32 or t.shape != (B,) or not t.is_contiguous()
            or t.get_device() != device.index):
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of B = {B} entries on {device}")
    return t.data_ptr()


def _slopes(alibi_slopes, Hq, device):
    """Device pointer of the fp32 [Hq] distance slopes (None stays None)."""
    import torch
    if alibi_slopes is None:
        return None
    if (not alibi_slopes.is_cuda or alibi_slopes.dtype is not torch.float32 or alibi_slopes.get_device() != device.index
            or alibi_slopes.shape != (Hq,) or not alibi_slopes.is_contiguous()):
        raise ValueError(f"alibi_slopes must be a contiguous fp32 CUDA tensor of Hq = {Hq} entries on {device}")
    return alibi_slopes.data_ptr()


def _same_device(first, *others):
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"all tensors must be on one device ({t.device} is not {first.device})")


def _out(t, name, shape, dtype, like):
    """`t`, checked to be a tensor of that shape on like's device, or a new one."""
    import torch
    if t is None:  # (empty_like takes 1.1 us less than new_empty with a type)
        return torch.empty_like(like) if dtype is like.dtype and like.shape == shape else like.new_empty(shape, dtype=dtype)
    if not t.is_cuda or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor {list(shape)}")
    _same_device(like, t)
    return t


@functools.lru_cache(maxsize=1024)
def _plan(which, device_index, B, Hq, Hkv, Nq, keys, d, num_splits):
    """(splits, workspace bytes) of a decode with changed scores ("score") or over a 4-bit cache
    ("kv4"): the sizes decide, on the current device."""
    splits, nbytes = ((fa_decode_score_num_splits, fa_decode_score_workspace_bytes) if which == "score"
                      else (fa_decode_kv4_num_splits, fa_decode_kv4_workspace_bytes))
    if num_splits is None:
        num_splits = splits(B, Hq, Hkv, Nq, keys, d)
        if num_splits < 1:
            raise FAError(FA_ERR_GQA if Hq % Hkv else FA_ERR_UNSUPPORTED, splits.__name__)
    return num_splits, nbytes(B, Hq, Hkv, Nq, keys, d, num_splits)


def _key_range(key_range, B, N, device):
    """Device pointer of the int32 [B, N, 2] key ranges (None stays None)."""
    import torch
    if key_range is None:
        return None
    if (not key_range.is_cuda or key_range.dtype is not torch.int32 or key_range.get_device() != device.index
            or key_range.shape != (B, N, 2) or not key_range.is_contiguous()):
        raise ValueError(f"key_range must be a contiguous int32 CUDA tensor [{B}, {N}, 2] on {device}")
    return key_range.data_ptr()


def _changes_scores(softcap, alibi_slopes, key_range=None):
    return bool(softcap) or alibi_slopes is not None or key_range is not None


def _score_alone(win, dropout_p, block_mask):
    if win is not None or dropout_p or block_mask is not None:
        raise ValueError("softcap, alibi_slopes and key_range combine with causal only "
                         "(no window, dropout or block_mask; a window is a key_range)")


def fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
        window=None, dropout_p: float = 0.0, seed: int = 0, block_mask=None, softcap: float = 0.0,
        alibi_slopes=None, key_range=None):
    """O, LSE = attention(q, k, v); q [B,Hq,N,d], k/v [B,Hkv,N,d] bf16 on one GPU.
    ``window=(left, right)``: local attention, key j visible to query i iff
    i - left <= j <= i + right (-1 = unlimited on that side).  ``dropout_p`` > 0: attention
    dropout with the Philox4x32-10 mask of ``seed`` (full or causal attention).
    ``block_mask``: block-sparse attention, uint8 (or bool) [B, Hq, ceil(N/128), ceil(N/128)]
    on the GPU, nonzero = the 128 x 128 block is computed (with or without ``causal``).
    Changed scores (with or without ``causal``): ``softcap`` c > 0 makes each scaled score x
    c tanh(x / c); ``alibi_slopes`` fp32 [Hq] takes slope |i - j| off; ``key_range`` int32
    [B, N, 2] gives the keys lo <= j < hi that each query row sees (see document_ranges and
    prefix_ranges); a row without keys gets O = 0 and LSE = -inf."""
    import torch
    win = _window(causal, window)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n)
    B, Hq, Hkv, N, d = _dims(q, k)
    if v.shape != k.shape:
        raise ValueError("v must match k")
    scale = default_scale(d) if scale is None else scale
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if _changes_scores(softcap, alibi_slopes, key_range):
        _score_alone(win, dropout_p, block_mask)
        _same_device(q, k, v)
        if out is not None:
            _out(o, "out", q.shape, torch.bfloat16, q)
        if lse is not None:
            _out(l, "lse", (B, Hq, N), torch.float32, q)
        with _on(q):
            fa_fwd_score(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                         _slopes(alibi_slopes, Hq, q.device), _key_range(key_range, B, N, q.device),
                         B, Hq, Hkv, N, d, causal, softcap, scale, _stream_handle(q))
        return o, l
    bm = _block_mask(block_mask, B, Hq, N, win, dropout_p)
    if bm is not None:
        fa_fwd_blocksparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                           bm.data_ptr(), B, Hq, Hkv, N, d, causal, scale, _stream_handle(q))
    elif dropout_p:
        if win is not None:
            raise ValueError("dropout is supported with full or causal attention only")
        fa_fwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                       B, Hq, Hkv, N, d, causal, dropout_p, seed, scale, _stream_handle(q))
    elif win is None:
        fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
               B, Hq, Hkv, N, d, causal, scale, _stream_handle(q))
    else:
        fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                      B, Hq, Hkv, N, d, win[0], win[1], scale, _stream_handle(q))
    return o, l


def bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
        workspace=None, dq=None, dk=None, dv=None, window=None, dropout_p: float = 0.0,
        seed: int = 0, block_mask=None, softcap: float = 0.0, alibi_slopes=None, key_range=None):
    """dQ, dK, dV of <O, dO> given the forward's O and LSE (same causal / window /
    dropout / block_mask / softcap / alibi_slopes / key_range; the last two are constants
    without a gradient)."""
    import torch
    win = _window(causal, window)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, n)
    B, Hq, Hkv, N, d = _dims(q, k)
    scale = default_scale(d) if scale is None else scale
    score = _changes_scores(softcap, alibi_slopes, key_range)
    nbytes = (fa_bwd_score_workspace_bytes if score else fa_bwd_workspace_bytes)(B, Hq, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
            dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), B, Hq, Hkv, N, d)
    if score:
        _score_alone(win, dropout_p, block_mask)
        _same_device(q, k, workspace)
        for t, n, like in ((v, "v", k), (o, "o", q), (dout, "dout", q), (dq, "dq", q), (dk, "dk", k), (dv, "dv", k)):
            _out(t, n, like.shape, torch.bfloat16, q)
        _out(lse, "lse", (B, Hq, N), torch.float32, q)
        with _on(q):
            fa_bwd_score(*ptrs[:11], _slopes(alibi_slopes, Hq, q.device),
                         _key_range(key_range, B, N, q.device), *ptrs[11:], causal, softcap, scale,
                         _stream_handle(q))
        return dq, dk, dv
    bm = _block_mask(block_mask, B, Hq, N, win, dropout_p)
    if bm is not None:
        fa_bwd_blocksparse(*ptrs[:11], bm.data_ptr(), *ptrs[11:], causal, scale, _stream_handle(q))
    elif dropout_p:
        if win is not None:
            raise ValueError("dropout is supported with full or causal attention only")
        fa_bwd_dropout(*ptrs, causal, dropout_p, seed, scale, _stream_handle(q))
    elif win is None:
        fa_bwd(*ptrs, causal, scale, _stream_handle(q))
    else:
        fa_bwd_window(*ptrs, win[0], win[1], scale, _stream_handle(q))
    return dq, dk, dv


def decode(q, k, v, seqlens_k=None, causal: bool = False, scale: float | None = None,
           num_splits: int | None = None, out=None, lse=None, workspace=None, softcap: float = 0.0,
           alibi_slopes=None):
    """Attention of q [B, Hq, Nq, d] against a cache k, v [B, Hkv, Nk, d] (bf16, one GPU),
    of which the first seqlens_k[b] keys are valid (int32 [B] on the GPU, or None: all).
    Causal: the Nq queries are the last Nq positions.  ``softcap`` and ``alibi_slopes`` change
    the scores as in fwd, the new rows at the last Nq positions.  Returns (O, LSE); rows that
    see no key get O = 0 and LSE = -inf."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n)
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("expected q [B,Hq,Nq,d] and k, v [B,Hkv,Nk,d]")
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if (Bk, dk) != (B, d):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)}")
    lens_ptr = None
    if seqlens_k is not None:
        if (not seqlens_k.is_cuda or seqlens_k.dtype != torch.int32 or seqlens_k.numel() != B
                or not seqlens_k.is_contiguous()):
            raise ValueError("seqlens_k must be a contiguous int32 CUDA tensor of B entries")
        lens_ptr = seqlens_k.data_ptr()
    scale = default_scale(d) if scale is None else scale
    if _changes_scores(softcap, alibi_slopes):
        _same_device(q, k, v, seqlens_k, workspace)
        with _on(q):
            num_splits, nbytes = _plan("score", q.device.index, B, Hq, Hkv, Nq, Nk, d, num_splits)
            if workspace is None and nbytes > 0:
                workspace = q.new_empty(nbytes, dtype=torch.uint8)
            o = _out(out, "out", q.shape, torch.bfloat16, q)
            l = _out(lse, "lse", (B, Hq, Nq), torch.float32, q)
            fa_decode_score(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(), lens_ptr,
                            _slopes(alibi_slopes, Hq, q.device), None if workspace is None else workspace.data_ptr(),
                            0 if workspace is None else workspace.numel() * workspace.element_size(),
                            B, Hq, Hkv, Nq, Nk, d, causal, num_splits, softcap, scale, _stream_handle(q))
        return o, l
    if num_splits is None:
        num_splits = fa_decode_num_splits(B, Hq, Hkv, Nq, Nk, d)
        if num_splits < 1:
            raise FAError(FA_ERR_UNSUPPORTED, "fa_decode_num_splits")
    nbytes = fa_decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    fa_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(), lens_ptr,
              ws_ptr, ws_bytes, B, Hq, Hkv, Nq, Nk, d, causal, num_splits, scale,
              _stream_handle(q))
    return o, l


def document_ranges(cu_seqlens, N: int):
    """key_range [B, N, 2] of rows packed with documents: cu_seqlens int32 or int64 [B, D + 1],
    the ascending offsets of the D documents of each row (repeat the last one for rows with
    fewer).  Positions outside every document see no key."""
    import torch
    pos = torch.arange(N, device=cu_seqlens.device)
    at = torch.searchsorted(cu_seqlens.contiguous(), pos.to(cu_seqlens.dtype).repeat(cu_seqlens.shape[0], 1),
                            right=True)
    inside = (at > 0) & (at < cu_seqlens.shape[1])
    end = at.clamp(1, cu_seqlens.shape[1] - 1)
    lo = torch.where(inside, cu_seqlens.gather(1, end - 1), torch.zeros_like(cu_seqlens[:, :1]))
    hi = torch.where(inside, cu_seqlens.gather(1, end), torch.zeros_like(cu_seqlens[:, :1]))
    return torch.stack((lo, hi), -1).to(torch.int32)


def prefix_ranges(prefix_lens, N: int):
    """key_range [B, N, 2] of rows whose first prefix_lens[b] keys are visible to every query and
    the others causally (call without ``causal``)."""
    import torch
    hi = torch.maximum(torch.arange(1, N + 1, device=prefix_lens.device), prefix_lens[:, None]).clamp(max=N)
    return torch.stack((torch.zeros_like(hi), hi), -1).to(torch.int32)


#: A key/value cache held in 4 bits (see fa_kv4_write in include/fa.h for the format):
#: uint8 [B, Hkv, cap, d/2] codes and fp16 [B, Hkv, cap, 2 d/32] params of K and of V.
KV4Cache = collections.namedtuple("KV4Cache", "k_codes k_params v_codes v_params")


def kv4_alloc(B: int, Hkv: int, cap: int, d: int, device="cuda"):
    """An empty 4-bit cache for `cap` tokens (a multiple of 64).  Its memory is not
    initialised: only what kv4_write wrote may be read or attended to."""
    import torch
    if d not in (64, 128, 256) or cap < 1 or cap % 64 or B < 1 or Hkv < 1:
        raise ValueError("kv4_alloc needs B, Hkv >= 1, cap a multiple of 64 and d in {64, 128, 256}")
    codes = lambda: torch.empty((B, Hkv, cap, d // 2), dtype=torch.uint8, device=device)
    params = lambda: torch.empty((B, Hkv, cap, d // 16), dtype=torch.float16, device=device)
    return KV4Cache(codes(), params(), codes(), params())


def _kv4(cache):
    """(B, Hkv, cap, d) of a cache, after checking its four tensors."""
    import torch
    kc, kp, vc, vp = cache
    if kc.dim() != 4:
        raise ValueError("cache codes must be [B, Hkv, cap, d/2]")
    shape, dev = kc.shape, kc.get_device()
    B, Hkv, cap, half = shape
    par = (B, Hkv, cap, half // 8)
    if not (kc.is_cuda and kp.get_device() == dev and vc.get_device() == dev and vp.get_device() == dev
            and kc.dtype is vc.dtype is torch.uint8 and kp.dtype is vp.dtype is torch.float16
            and vc.shape == shape and kp.shape == par and vp.shape == par and kc.is_contiguous()
            and kp.is_contiguous() and vc.is_contiguous() and vp.is_contiguous()):
        raise ValueError(f"a cache holds contiguous CUDA tensors of one device: uint8 codes {list(shape)} and "
                         f"float16 params {list(par)}, of K and of V")
    return B, Hkv, cap, 2 * half


def _pointers(cache):
    kc, kp, vc, vp = cache
    return kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr()


def kv4_write(cache, k, v, start=None, counts=None) -> None:
    """Quantise new tokens k, v [B, Hkv, n, d] bf16 into positions start[b] .. start[b]+n-1 of
    the cache (int32 [B] on the GPU, or None: 0); with counts (int32 [B]) only the first
    counts[b] of them.  Positions outside the cache are skipped and reported by
    fa_device_status as FA_ERR_SEQLENS."""
    B, Hkv, cap, d = _kv4(cache)
    _need(k, "k")
    _need(v, "v")
    n = k.shape[2] if k.dim() == 4 else 0
    if v.shape != k.shape or k.shape != (B, Hkv, n, d):
        raise ValueError(f"expected k and v [{B}, {Hkv}, n, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    _same_device(cache.k_codes, k, v)
    sp, cp = _int32_vector(start, "start", B, k.device), _int32_vector(counts, "counts", B, k.device)
    if n == 0:
        return
    with _on(k):
        fa_kv4_write(k.data_ptr(), v.data_ptr(), *_pointers(cache), sp, cp, B, Hkv, n, cap, d,
                     _stream_handle(k))


def kv4_read(cache, n: int, start=None, k=None, v=None):
    """K, V [B, Hkv, n, d] bf16: what positions start[b] .. start[b]+n-1 of the cache stand for
    (int32 [B] on the GPU, or None: 0)."""
    import torch
    B, Hkv, cap, d = _kv4(cache)
    n = int(n)
    if n < 0:
        raise ValueError("n must not be negative")
    k = _out(k, "k", (B, Hkv, n, d), torch.bfloat16, cache.k_codes)
    v = _out(v, "v", (B, Hkv, n, d), torch.bfloat16, k)
    sp = _int32_vector(start, "start", B, cache.k_codes.device)
    if n > 0:
        with _on(k):
            fa_kv4_read(*_pointers(cache), k.data_ptr(), v.data_ptr(), sp, B, Hkv, n, cap,
                        d, _stream_handle(k))
    return k, v


def decode_kv4(q, cache, seqlens_k=None, causal: bool = False, scale: float | None = None,
               softcap: float = 0.0, alibi_slopes=None, num_splits: int | None = None, out=None,
               lse=None, workspace=None):
    """Attention of q [B, Hq, Nq, d] bf16 against a 4-bit cache (KV4Cache), of which the first
    seqlens_k[b] tokens are valid (int32 [B] on the GPU, or None: all).  Causal: the Nq queries
    are the last Nq positions.  softcap c > 0: scores c tanh(x / c); alibi_slopes fp32 [Hq]:
    slope |i - j| taken off.  Returns (O, LSE); rows that see no key get O = 0, LSE = -inf."""
    import torch
    B, Hkv, cap, d = _kv4(cache)
    _need(q, "q")
    if q.dim() != 4 or q.shape[0] != B or q.shape[3] != d:
        raise ValueError(f"expected q [{B}, Hq, Nq, {d}], got {tuple(q.shape)}")
    _, Hq, Nq, _ = q.shape
    _same_device(q, cache.k_codes, workspace)
    dev = q.device
    lens_ptr = _int32_vector(seqlens_k, "seqlens_k", B, dev)
    slopes_ptr = _slopes(alibi_slopes, Hq, dev)
    scale = default_scale(d) if scale is None else scale
    with _on(q):
        num_splits, nbytes = _plan("kv4", dev.index, B, Hq, Hkv, Nq, cap, d, num_splits)
        if workspace is None and nbytes > 0:
            workspace = q.new_empty(nbytes, dtype=torch.uint8)
        o = _out(out, "out", q.shape, torch.bfloat16, q)
        l = _out(lse, "lse", (B, Hq, Nq), torch.float32, q)
        ws_ptr = None if workspace is None else workspace.data_ptr()
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        fa_decode_kv4(q.data_ptr(), *_pointers(cache), o.data_ptr(), l.data_ptr(), lens_ptr,
                      slopes_ptr, ws_ptr, ws_bytes, B, Hq, Hkv, Nq, cap, d, causal, num_splits, softcap,
                      scale, _stream_handle(q))
    return o, l


def merge(o_parts, lse_parts, out=None, lse=None):
    """Combine partial results over disjoint key sets: o_parts [S, ..., d] fp32 (each part
    normalised), lse_parts [S, ...] fp32 -> (O bf16 [..., d], LSE fp32 [...])."""
    import torch
    if (not o_parts.is_cuda or o_parts.dtype != torch.float32 or not o_parts.is_contiguous()
            or not lse_parts.is_cuda or lse_parts.dtype != torch.float32
            or not lse_parts.is_contiguous() or tuple(lse_parts.shape) != tuple(o_parts.shape[:-1])):
        raise ValueError("o_parts [S, ..., d] and lse_parts [S, ...] must be contiguous fp32 CUDA tensors")
    S, d = o_parts.shape[0], o_parts.shape[-1]
    rows = lse_parts[0].numel()
    o = torch.empty(o_parts.shape[1:], dtype=torch.bfloat16, device=o_parts.device) if out is None else out
    l = torch.empty(lse_parts.shape[1:], dtype=torch.float32, device=o_parts.device) if lse is None else lse
    fa_merge(o_parts.data_ptr(), lse_parts.data_ptr(), o.data_ptr(), l.data_ptr(), S, rows, d,
             _stream_handle(o_parts))
    return o, l


def _varlen_args(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, window):
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n)
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or q.shape[2] != k.shape[2]:
        raise ValueError("expected q [total_q, Hq, d] and k, v [total_k, Hkv, d]")
    for c, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k")):
        if not c.is_cuda or c.dtype != torch.int32 or not c.is_contiguous() or c.dim() != 1:
            raise ValueError(f"{n} must be a contiguous int32 CUDA vector of B + 1 offsets")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both hold B + 1 >= 2 offsets")
    if window is not None and causal:
        raise ValueError("give either causal=True or window=(left, right), not both")
    left, right = (int(w) for w in window) if window is not None else (-1, 0 if causal else -1)
    return (cu_seqlens_q.numel() - 1, q.shape[1], k.shape[1], q.shape[0], k.shape[0],
            int(max_seqlen_q), int(max_seqlen_k), q.shape[2], left, right)


def fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
               causal: bool = False, scale: float | None = None, window=None, out=None, lse=None):
    """Attention over packed sequences: q [total_q, Hq, d], k/v [total_k, Hkv, d] bf16,
    cu_seqlens_* int32 [B+1] on the GPU.  Returns O [total_q, Hq, d] and LSE [total_q, Hq].
    causal / window bands are aligned to the end of each sequence."""
    import torch
    B, Hq, Hkv, tq, tk, mq, mk, d, left, right = _varlen_args(
        q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, window)
    scale = default_scale(d) if scale is None else scale
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((tq, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                  cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Hq, Hkv, tq, tk, mq, mk, d,
                  left, right, scale, _stream_handle(q))
    return o, l


def bwd_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
               causal: bool = False, scale: float | None = None, window=None, workspace=None,
               dq=None, dk=None, dv=None):
    """dQ, dK, dV of <O, dO> for packed sequences (same arguments as fwd_varlen)."""
    import torch
    B, Hq, Hkv, tq, tk, mq, mk, d, left, right = _varlen_args(
        q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, window)
    _need(o, "o")
    _need(dout, "dout")
    scale = default_scale(d) if scale is None else scale
    nbytes = fa_bwd_varlen_workspace_bytes(Hq, tq, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    fa_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                  dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                  cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Hq, Hkv, tq, tk, mq, mk, d,
                  left, right, scale, _stream_handle(q))
    return dq, dk, dv
