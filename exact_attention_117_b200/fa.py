"""Python binding of the C ABI in include/fa.h (argument marshalling only).

Every step of the computation runs in the CUDA library ``libfa_b200.so``; this
module only checks tensor properties, takes device pointers and the current
stream from torch, and turns status codes into exceptions (through ctypes, the
rotary and 4-bit cache calls through the extension module of csrc/binding.cpp).
There is no fallback: if the library is missing or not built for this GPU, every
call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FA_LIBRARY selects another build of the same library (e.g. the bounds-checked
# libfa_b200_debug.so); by default the release build next to this file.
LIB_PATH = os.environ.get("FA_LIBRARY") or os.path.join(_HERE, "libfa_b200.so")

FA_OK = 0
STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_SHAPE", 3: "FA_ERR_UNSUPPORTED_D",
    4: "FA_ERR_ALIGN", 5: "FA_ERR_SCALE", 6: "FA_ERR_WORKSPACE", 7: "FA_ERR_CUDA",
    8: "FA_ERR_DEVICE_TIMEOUT", 9: "FA_ERR_STATE", 10: "FA_ERR_PAGE",
}
KERNELS = ("fwd", "bwd_pre", "bwd_main", "bwd_dq", "fwd_combine", "fwd_kv_outer", "rotary",
           "kv4_plan", "kv4_append", "kv4_gather", "kv4_attend", "kv4_combine")

_lib = None
_native = None  # the extension module of csrc/binding.cpp, bound to _lib


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.fa_status_string(status).decode() if _lib is not None else ""
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({msg})")


def load() -> ctypes.CDLL:
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.restype = i
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.fa_fwd_splitkv_workspace_size.restype = sz
    lib.fa_fwd_splitkv_workspace_size.argtypes = [i, i, i, i, i]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_fwd_kv_outer_workspace_size.restype = sz
    lib.fa_fwd_kv_outer_workspace_size.argtypes = [i, i, i, i]
    lib.fa_fwd_kv_outer.restype = i
    lib.fa_fwd_kv_outer.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]
    lib.fa_bwd_workspace_size.restype = sz
    lib.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa_bwd.restype = i
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, f, vp]
    lib.fa_bwd_deterministic.restype = i
    lib.fa_bwd_deterministic.argtypes = lib.fa_bwd.argtypes
    lib.fa_bwd_noalloc.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    ll = ctypes.c_longlong
    lib.fa_rotary.restype = i
    lib.fa_rotary.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp, vp, i, ll, vp, i, i, f, i, i, vp]
    lib.fa_kv4_cache_size.restype = sz
    lib.fa_kv4_cache_size.argtypes = [i, i, i, i]
    lib.fa_kv4_plan.restype = i
    lib.fa_kv4_plan.argtypes = [vp, vp, vp, ll, i, vp, i, vp, i, i, i, vp, vp, vp, vp, vp, vp, vp]
    lib.fa_kv4_append.restype = i
    lib.fa_kv4_append.argtypes = [vp, vp, vp, vp, ll, i, i, i, i, vp, vp]
    lib.fa_kv4_gather.restype = i
    lib.fa_kv4_gather.argtypes = [vp, vp, vp, vp, ll, i, i, i, i, vp, vp]
    lib.fa_kv4_attention_workspace_size.restype = sz
    lib.fa_kv4_attention_workspace_size.argtypes = [i, i, i, i]
    lib.fa_kv4_attention.restype = i
    lib.fa_kv4_attention.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, ll, vp, i,
                                     i, f, i, vp, sz, vp]
    lib.fa_check_device_error.restype = i
    lib.fa_check_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
    lib.fa_selftest_watchdog.restype = i
    lib.fa_selftest_watchdog.argtypes = [ctypes.c_uint, vp]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_status_string.argtypes = [i]
    lib.fa_timing_begin.restype = i
    lib.fa_timing_begin.argtypes = []
    lib.fa_timing_end.restype = i
    lib.fa_timing_end.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int)]
    lib.fa_version.restype = i
    lib.fa_version.argtypes = []
    _lib = lib
    return lib


def _load_native():
    """The extension module with the serving calls, bound to the loaded library
    (raises if it has not been built)."""
    global _native
    if _native is None:
        lib = load()
        path = os.path.join(_HERE, "_fa_binding.so")
        if not os.path.exists(path):
            raise RuntimeError(f"binding not built: {path} is missing "
                               "(run __graft_entry__.build())")
        from . import build
        if build.binding_built_for() not in ("", build.binding_target()):  # ("": not said)
            raise RuntimeError(f"{path} was built for another torch or Python "
                               "(run __graft_entry__.build())")
        spec = importlib.util.spec_from_file_location("_fa_binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.fa_rotary, lib.fa_kv4_plan, lib.fa_kv4_append, lib.fa_kv4_gather,
            lib.fa_kv4_attention_workspace_size, lib.fa_kv4_attention)))
        _native = module
    return _native


def _check(status: int, where: str):
    if status != FA_OK:
        raise FaError(status, where)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_qkv(*ts: torch.Tensor):
    ref = ts[0]
    if ref.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    for t in ts:
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("tensors must be contiguous bf16 CUDA tensors")
        if t.shape != ref.shape:
            raise ValueError("all tensors must have the same [B, H, N, d] shape")


def fwd_raw(q: int, k: int, v: int, o: int, lse: int, B: int, H: int, N: int, d: int,
            causal: bool, scale: float, stream: int) -> int:
    """Direct call of ``fa_fwd`` with raw pointers; returns the status code."""
    return load().fa_fwd(q, k, v, o, lse, B, H, N, d, int(bool(causal)), float(scale), stream)


def bwd_raw(q, k, v, o, lse, do, dq, dk, dv, ws, ws_bytes, B, H, N, d, causal, scale,
            stream) -> int:
    """Direct call of ``fa_bwd`` with raw pointers; returns the status code."""
    return load().fa_bwd(q, k, v, o, lse, do, dq, dk, dv, ws, ws_bytes, B, H, N, d,
                         int(bool(causal)), float(scale), stream)


def workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_size(B, H, N, d))


def forward(q, k, v, causal: bool = False, scale: Optional[float] = None, out=None,
            lse=None, stream=None):
    """O, LSE = attention(q, k, v); all [B, H, N, d] bf16 on the GPU."""
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check(fwd_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d, causal, scale,
                   _stream_ptr(stream)), "fa_fwd")
    return out, lse


def splitkv_workspace_size(B: int, H: int, N: int, d: int, num_splits: int) -> int:
    return int(load().fa_fwd_splitkv_workspace_size(B, H, N, d, num_splits))


def forward_splitkv(q, k, v, causal: bool = False, scale: Optional[float] = None,
                    num_splits: int = 2, out=None, lse=None, workspace=None, stream=None):
    """O, LSE through the split-KV forward (key range cut into ``num_splits``)."""
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = splitkv_workspace_size(B, H, N, d, num_splits)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(load().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                                 int(bool(causal)), float(scale), int(num_splits),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream)), "fa_fwd_splitkv")
    return out, lse


def bwd_deterministic_raw(q, k, v, o, lse, do, dq, dk, dv, ws, ws_bytes, B, H, N, d, causal,
                          scale, stream) -> int:
    """Direct call of ``fa_bwd_deterministic`` with raw pointers; returns the status code."""
    return load().fa_bwd_deterministic(q, k, v, o, lse, do, dq, dk, dv, ws, ws_bytes, B, H, N, d,
                                       int(bool(causal)), float(scale), stream)


def kv_outer_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_fwd_kv_outer_workspace_size(B, H, N, d))


def forward_kv_outer(q, k, v, causal: bool = False, scale: Optional[float] = None, out=None,
                     lse=None, workspace=None, stream=None):
    """O, LSE through the KV-outer (FlashAttention-1 order) forward kernel."""
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = kv_outer_workspace_size(B, H, N, d)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(load().fa_fwd_kv_outer(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                                  int(bool(causal)), float(scale), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  _stream_ptr(stream)), "fa_fwd_kv_outer")
    return out, lse


def backward(q, k, v, o, lse, do, causal: bool = False, scale: Optional[float] = None,
             dq=None, dk=None, dv=None, workspace=None, stream=None,
             deterministic: bool = False):
    """dQ, dK, dV of sum(dO * O); the fp32 workspace is allocated here if not given.

    ``deterministic=True`` calls ``fa_bwd_deterministic`` (dQ summed in a fixed
    order, bitwise reproducible) instead of ``fa_bwd`` (dQ summed by atomics)."""
    _check_qkv(q, k, v, o, do)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    need = workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    raw, name = (bwd_deterministic_raw, "fa_bwd_deterministic") if deterministic else \
        (bwd_raw, "fa_bwd")
    _check(raw(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
               _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
               B, H, N, d, causal, scale, _stream_ptr(stream)), name)
    return dq, dk, dv


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # FA_BWD_NOALLOC_SCRATCH_BYTES in include/fa.h


def bwd_noalloc_raw(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d, causal, scale,
                    stream) -> int:
    """Direct call of ``fa_bwd_noalloc`` with raw pointers; returns the status code."""
    return load().fa_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d,
                                 int(bool(causal)), float(scale), stream)


def backward_noalloc(q, k, v, o, lse, do, causal: bool = False, scale: Optional[float] = None,
                     dq=None, dk=None, dv=None, stream=None):
    """Like ``backward`` but through ``fa_bwd_noalloc``: the library's own fixed
    scratch array replaces the workspace, so the C call allocates nothing.
    Problems needing more than ``NOALLOC_SCRATCH_BYTES`` of scratch raise
    FaError(FA_ERR_WORKSPACE).  (The outputs are allocated here by torch only if
    the caller does not pass them.)"""
    _check_qkv(q, k, v, o, do)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    _check(bwd_noalloc_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                           _ptr(dk), _ptr(dv), B, H, N, d, causal, scale, _stream_ptr(stream)),
           "fa_bwd_noalloc")
    return dq, dk, dv


# ------------------------------------------------------------ rotary positions
def _stream_arg(stream):
    return None if stream is None else int(stream.cuda_stream)


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, factor: float = 1.0,
                       original_length: Optional[int] = None, fast_turns: float = 32.0,
                       slow_turns: float = 1.0, device="cuda"):
    """``inv_freq`` (fp64 ``[rotary_dim / 2]``, radians per position) and the
    amplitude for :func:`rotary`.

    Pair ``i`` turns by ``base ** (-2 i / rotary_dim)``.  With a context
    ``factor`` above 1 positions are interpolated: by ``factor`` in every pair
    or, given the ``original_length``, only in the pairs that turn fewer than
    ``slow_turns`` times in it, not at all in those that turn more than
    ``fast_turns`` times, in proportion to their turns between; the amplitude is
    then ``0.1 ln(factor) + 1``.  (A model whose ramp runs over the pairs' index, the
    logarithm of the turns, has other frequencies between: pass its own.)"""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not (factor >= 1.0 and base > 0.0 and fast_turns > slow_turns):
        raise ValueError("factor >= 1, base > 0 and fast_turns > slow_turns are required")
    f = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    amplitude = 1.0
    if factor > 1.0 and original_length is None:
        f = f / factor
    elif factor > 1.0:
        turns = original_length * f / (2.0 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    return f.to(device), amplitude


def rotary(q, k, positions, inv_freq, interleaved: bool = False, amplitude: float = 1.0,
           out_q=None, out_k=None, stream=None):
    """Rotary positions of queries ``[B, H, N, d]`` and keys ``[B, Hk, N, d]``
    (or ``None``), bf16, fp16 or fp32 with any strides but a contiguous ``d``:
    packed ``[tokens, heads, d]`` goes in as ``x.transpose(0, 1)[None]``.
    ``positions``: int32 or int64 ``[N]`` or ``[B, N]``.  The first
    ``2 * len(inv_freq)`` channels turn, in pairs ``(i, i + len(inv_freq))`` or,
    ``interleaved``, ``(2i, 2i + 1)``.  Outputs may be the inputs.  Like every call
    here it records nothing for autograd: the gradient is :func:`rotary_backward`."""
    st, out_q, out_k = (_native or _load_native()).rotary(
        q, k, positions, inv_freq, interleaved, amplitude, out_q, out_k, _stream_arg(stream), False)
    if st:
        raise FaError(st, "fa_rotary")
    return out_q, out_k


def rotary_backward(dq, dk, positions, inv_freq, interleaved: bool = False,
                    amplitude: float = 1.0, out_q=None, out_k=None, stream=None):
    """Gradients of :func:`rotary`'s inputs from those of its outputs (the same
    arguments otherwise)."""
    st, out_q, out_k = (_native or _load_native()).rotary(
        dq, dk, positions, inv_freq, interleaved, amplitude, out_q, out_k, _stream_arg(stream), True)
    if st:
        raise FaError(st, "fa_rotary")
    return out_q, out_k


# ------------------------------------------------------------ 4-bit KV cache
class Kv4Plan(NamedTuple):
    lengths: torch.Tensor     # int32 [requests]
    cu_tokens: torch.Tensor   # int32 [requests + 1]
    slots: torch.Tensor       # int64 [max_tokens]
    positions: torch.Tensor   # int32 [max_tokens]
    status: torch.Tensor      # int32 [1]: 0, or what refused the step
    free_range: torch.Tensor  # int64 [2]


def kv4_cache(pages: int, kv_heads: int, page_size: int, d: int, device="cuda"):
    """An empty 4-bit cache ``uint8 [pages, kv_heads, page_size / 16, 18 d]``."""
    if not load().fa_kv4_cache_size(pages, kv_heads, page_size, d):
        raise ValueError("pages and kv_heads >= 1, page_size a multiple of 16, d 64 or 128")
    return torch.zeros((pages, kv_heads, page_size // 16, 18 * d), dtype=torch.uint8,
                       device=device)


def kv4_plan(lengths, new_lengths, block_table, free_pages, free_range, page_size: int,
             max_tokens: int, lengths_out=None, free_range_out=None, stream=None) -> Kv4Plan:
    """Pages, slots and positions of a step, on the device: requests go from
    ``lengths`` (int32 ``[requests]``) to ``new_lengths``.  ``block_table``
    (int32 ``[requests, width]``) and ``free_pages`` (int32 ring, live from
    ``free_range[0]`` to ``free_range[1]``, int64) are updated in place;
    lengths and range too if they are passed as their own outputs.  The tensors that
    the call makes share one allocation, which lives as long as any of them.  See
    ``fa_kv4_plan`` in include/fa.h for the statuses."""
    st, *out = (_native or _load_native()).plan(
        lengths, new_lengths, block_table, free_pages, free_range, page_size, max_tokens,
        lengths_out, free_range_out, _stream_arg(stream))
    if st:
        raise FaError(st, "fa_kv4_plan")
    return Kv4Plan(*out)


def kv4_append(k, v, cache, slots, stream=None):
    """Quantises keys and values (bf16 ``[tokens, kv_heads, d]``, d contiguous)
    into ``slots`` (int64, ``page * page_size + place``; -1 skips, and no slot
    twice) of the cache."""
    st = (_native or _load_native()).append(k, v, cache, slots, _stream_arg(stream))
    if st:
        raise FaError(st, "fa_kv4_append")


def kv4_gather(cache, slots, out_k=None, out_v=None, stream=None):
    """The values that the cache holds for ``slots``: bf16 keys and values
    ``[tokens, kv_heads, d]``; zeros for slots outside the cache."""
    st, out_k, out_v = (_native or _load_native()).gather(cache, slots, out_k, out_v,
                                                          _stream_arg(stream))
    if st:
        raise FaError(st, "fa_kv4_gather")
    return out_k, out_v


def kv4_attention_workspace_size(heads: int, kv_heads: int, d: int, max_tokens: int) -> int:
    return int(load().fa_kv4_attention_workspace_size(heads, kv_heads, d, max_tokens))


def kv4_attention(q, cache, block_table, lengths, cu_tokens, max_tokens: int,
                  causal: bool = True, scale: Optional[float] = None, out=None, lse=None,
                  workspace=None, stream=None):
    """O ``[tokens, heads, d]``, LSE ``[tokens, heads]`` of packed queries (bf16
    or fp16 ``[tokens, heads, d]``, d contiguous) over the 4-bit cache.

    Request ``b``'s queries are rows ``cu_tokens[b] .. cu_tokens[b + 1]`` (int32)
    and the newest of its ``lengths[b]`` (int32) cached tokens; ``block_table``
    (int32 ``[requests, width]``) lists its pages.  ``max_tokens``: an upper
    bound on a request's query rows (it chooses the kernel).  Rows that see no
    key get zeros and -inf; rows of no request are left as they are.  What tokens
    hold that a row does not see changes none of its bits; the precision is
    ``fa_kv4_attention``'s in include/fa.h."""
    st, out, lse = (_native or _load_native()).attention(
        q, cache, block_table, lengths, cu_tokens, max_tokens, causal, scale, out, lse, workspace,
        _stream_arg(stream))
    if st:
        raise FaError(st, "fa_kv4_attention")
    return out, lse


def check_device_error(stream=None):
    """Synchronise and raise FaError if a kernel gave up on a bounded wait, or met
    a page index outside its cache."""
    detail = ctypes.c_uint(0)
    st = load().fa_check_device_error(_stream_ptr(stream), ctypes.byref(detail))
    if st != FA_OK:
        raise FaError(st, f"device error word 0x{detail.value:x}")


def selftest_watchdog(limit_ms: int = 200, stream=None):
    """Launch the bounded-wait self-test kernel (see fa_selftest_watchdog)."""
    _check(load().fa_selftest_watchdog(int(limit_ms), _stream_ptr(stream)), "fa_selftest_watchdog")


class KernelTimer:
    """Context manager: per-kernel CUDA-event time of every launch inside it."""

    def __enter__(self):
        _check(load().fa_timing_begin(), "fa_timing_begin")
        return self

    def __exit__(self, *exc):
        ms = (ctypes.c_float * len(KERNELS))()
        cnt = (ctypes.c_int * len(KERNELS))()
        _check(load().fa_timing_end(ms, cnt), "fa_timing_end")
        self.ms = {k: float(ms[i]) for i, k in enumerate(KERNELS)}
        self.launches = {k: int(cnt[i]) for i, k in enumerate(KERNELS)}
        return False
