"""Jet-Long dynamic bifocal RoPE attention for NVIDIA B200 -- Python binding.

Thin ctypes binding of ``libjetlong.so`` (C ABI declared in ``include/jetlong.h``).
Functions keep the C names without the ``jetlong_`` prefix.  This module only
marshals arguments: torch tensors supply device pointers and the current CUDA
stream; every step of the attention runs in the library's CUDA kernels.  There
is no fallback: if the library is missing the calls raise.

Method: "Jet-Long: Efficient Long-Context Extension with Dynamic Bifocal RoPE"
(gist.science/it/paper/2607.07740), Metodologia 1 (local window w0 with classic
RoPE; remote pairs at f(x) = floor(x/G), G = max(1, ceil(L/w_pretrained))) and
Metodologia 2 (rotations applied on the fly to an untouched cache; one exact
distance-routed softmax).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
from typing import NamedTuple

__all__ = [
    "BF16", "FP32", "JetLongError", "load_library", "group_size", "position_map", "prefill",
    "prefill_chunk", "prefill_varlen", "prefill_ie", "prefill_streamed", "decode_workspace_size",
    "decode", "decode_rope_cache", "decode_noalloc", "device_status", "last_error", "launch_count",
    "DECODE_NOALLOC_SCRATCH_BYTES", "selftest_wait_timeout", "debug_inject_timeout",
    "INJECT_PREFILL_KEY_TILE", "INJECT_DECODE_COPY", "debug_rope_phase", "debug_tile_plan", "debug_ex2", "debug_rope_keys",
    "BlockTables", "block_tables", "cache_append", "decode_tree_workspace_size", "decode_paged", "decode_tree",
    "tree_commit", "NO_PAGE",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libjetlong.so")

BF16 = 0
FP32 = 1
NO_PAGE = -2  # block table entry of rows that block_tables refused
_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT"}

_lock = threading.Lock()
_lib = None


class JetLongError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"jetlong {_STATUS.get(status, status)}: {message}")
        self.status = status


def load_library(path: str | None = None):
    """Load libjetlong.so (built in-tree by ``python -m rope_context_extension_jet_b200._build``)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with "
                               "`python -m rope_context_extension_jet_b200._build`")
        lib = ctypes.CDLL(p)
        vp, i32, i64, sz, dbl, flt = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                      ctypes.c_size_t, ctypes.c_double, ctypes.c_float)
        lib.jetlong_group_size.restype = i64
        lib.jetlong_group_size.argtypes = [i64, i64]
        lib.jetlong_position_map.restype = i32
        lib.jetlong_position_map.argtypes = [vp, i64, i64, vp]
        lib.jetlong_prefill.restype = i32
        lib.jetlong_prefill.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                        dbl, flt, i32, vp]
        lib.jetlong_prefill_ie_workspace_size.restype = sz
        lib.jetlong_prefill_ie_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.jetlong_prefill_ie.restype = i32
        lib.jetlong_prefill_ie.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, dbl, flt,
                                           i32, vp, sz, vp]
        lib.jetlong_prefill_streamed.restype = i32
        lib.jetlong_prefill_streamed.argtypes = [vp] * 8 + [i32, i32, i32, i32, i32, i32, i32, dbl, flt,
                                                            i32, i32, vp]
        lib.jetlong_prefill_varlen.restype = i32
        lib.jetlong_prefill_varlen.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, i32, i32,
                                               i32, dbl, flt, i32, vp]
        lib.jetlong_prefill_chunk.restype = i32
        lib.jetlong_prefill_chunk.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                              i32, i32, dbl, flt, i32, vp]
        lib.jetlong_decode_workspace_size.restype = sz
        lib.jetlong_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        for fn in (lib.jetlong_decode, lib.jetlong_decode_rope_cache):
            fn.restype = i32
            fn.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                           dbl, flt, i32, vp, sz, vp]
        lib.jetlong_decode_noalloc.restype = i32
        lib.jetlong_decode_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                               i32, dbl, flt, i32, vp]
        lib.jetlong_selftest_wait_timeout.restype = i32
        lib.jetlong_selftest_wait_timeout.argtypes = [vp]
        lib.jetlong_debug_inject_timeout.restype = i32
        lib.jetlong_debug_inject_timeout.argtypes = [i32, ctypes.c_longlong]
        lib.jetlong_debug_rope_phase.restype = i32
        lib.jetlong_debug_rope_phase.argtypes = [vp, i64, i32, dbl, i32, vp, vp]
        lib.jetlong_debug_tile_plan.restype = i32
        lib.jetlong_debug_tile_plan.argtypes = [i32, i32, i32, i32, vp, vp, vp]
        lib.jetlong_debug_ex2.restype = i32
        lib.jetlong_debug_ex2.argtypes = [vp, i64, vp, vp]
        lib.jetlong_debug_rope_keys.restype = i32
        lib.jetlong_debug_rope_keys.argtypes = [vp, i32, i32, i32, i32, dbl, vp, vp, ctypes.POINTER(ctypes.c_int), vp]
        lib.jetlong_block_tables.restype = i32
        lib.jetlong_block_tables.argtypes = [vp] * 13 + [i32] * 6 + [vp]
        lib.jetlong_cache_append.restype = i32
        lib.jetlong_cache_append.argtypes = [vp] * 5 + [i32] * 3 + [i64] * 4 + [i32] * 3 + [vp]
        lib.jetlong_decode_tree_workspace_size.restype = sz
        lib.jetlong_decode_tree_workspace_size.argtypes = [i32] * 5
        lib.jetlong_decode_paged.restype = i32
        lib.jetlong_decode_paged.argtypes = [vp] * 6 + [i32] * 9 + [dbl, flt, i32, vp, sz, vp]
        lib.jetlong_decode_tree.restype = i32
        lib.jetlong_decode_tree.argtypes = [vp] * 8 + [i32] * 11 + [dbl, flt, i32, vp, sz, vp]
        lib.jetlong_tree_commit.restype = i32
        lib.jetlong_tree_commit.argtypes = [vp] * 9 + [i32] * 9 + [vp]
        lib.jetlong_device_status.restype = i32
        lib.jetlong_device_status.argtypes = [vp]
        lib.jetlong_last_error.restype = ctypes.c_char_p
        lib.jetlong_last_error.argtypes = []
        lib.jetlong_launch_count.restype = ctypes.c_uint64
        lib.jetlong_launch_count.argtypes = []
        if path is None:
            _lib = lib
        return lib


def _check(status: int, lib=None):
    if status != 0:
        lib = lib or load_library()
        raise JetLongError(status, lib.jetlong_last_error().decode())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _dev(t, name):
    import torch
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device} but the library runs on the current device "
                         f"cuda:{torch.cuda.current_device()} (select it with torch.cuda.device)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _like(t, ref, name, ref_name):
    """The library writes ``t`` with ``ref``'s shape and element type."""
    if t.shape != ref.shape or t.dtype != ref.dtype:
        raise ValueError(f"{name} must match {ref_name}: shape {tuple(ref.shape)}, dtype {ref.dtype} "
                         f"(got {tuple(t.shape)}, {t.dtype})")


def _same_dtype(*named):
    if len({t.dtype for t, _ in named}) != 1:
        raise TypeError(", ".join(n for _, n in named) + " must share a dtype")


def last_error() -> str:
    return load_library().jetlong_last_error().decode()


def launch_count() -> int:
    return int(load_library().jetlong_launch_count())


def group_size(L: int, w_pretrained: int) -> int:
    """G = max(1, ceil(L / w_pretrained)); -1 for invalid arguments."""
    return int(load_library().jetlong_group_size(int(L), int(w_pretrained)))


def position_map(out, L: int, w_pretrained: int, stream=None):
    """Write floor(x / G) for x in [0, L) into the int32 CUDA tensor ``out``."""
    import torch
    if out.dtype != torch.int32 or out.numel() < L:
        raise ValueError("out must be an int32 tensor with at least L elements")
    lib = load_library()
    _check(lib.jetlong_position_map(_dev(out, "out"), int(L), int(w_pretrained), _stream(stream)),
           lib)
    return out


def prefill(q, k, v, out=None, *, w0: int, w_pretrained: int, rope_theta: float,
            scale: float | None = None, stream=None):
    """Routed causal attention over raw q [B,Hq,L,d], k/v [B,Hkv,L,d] (bf16 or fp32)."""
    import torch
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, L, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, L, d] matching q")
    _same_dtype((q, "q"), (k, "k"), (v, "v"))
    if out is None:
        out = torch.empty_like(q)
    _like(out, q, "out", "q")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    lib = load_library()
    _check(lib.jetlong_prefill(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"),
                               B, Hq, Hkv, L, d, int(w0), int(w_pretrained), float(rope_theta),
                               float(scale), _dtype_code(q), _stream(stream)), lib)
    return out


def prefill_chunk(q, kcache, vcache, P: int, out=None, *, w0: int, w_pretrained: int,
                  rope_theta: float, scale: float | None = None, stream=None):
    """Chunked prefill: raw queries q [B,Hq,C,d] at positions [P, P+C) over cache
    rows [0, P+C) of kcache/vcache [B,Hkv,Lcap,d]; G from P + C."""
    import torch
    B, Hq, C, d = q.shape
    _, Hkv, Lcap, _ = kcache.shape
    if vcache.shape != kcache.shape or kcache.shape[0] != B or kcache.shape[3] != d:
        raise ValueError("kcache and vcache must be [B, Hkv, Lcap, d] matching q")
    _same_dtype((q, "q"), (kcache, "kcache"), (vcache, "vcache"))
    if out is None:
        out = torch.empty_like(q)
    _like(out, q, "out", "q")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    lib = load_library()
    _check(lib.jetlong_prefill_chunk(_dev(q, "q"), _dev(kcache, "kcache"), _dev(vcache, "vcache"),
                                     _dev(out, "out"), B, Hq, Hkv, int(P), C, Lcap, d, int(w0),
                                     int(w_pretrained), float(rope_theta), float(scale),
                                     _dtype_code(q), _stream(stream)), lib)
    return out


def prefill_ie(q, k, v, out=None, *, w0: int, w_pretrained: int, rope_theta: float,
               scale: float | None = None, workspace=None, stream=None):
    """The pages' three-pass inclusion-exclusion form of the prefill (same
    result as ``prefill``; for comparing the two forms)."""
    import torch
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, L, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, L, d] matching q")
    _same_dtype((q, "q"), (k, "k"), (v, "v"))
    if out is None:
        out = torch.empty_like(q)
    _like(out, q, "out", "q")
    lib = load_library()
    need = int(lib.jetlong_prefill_ie_workspace_size(B, Hq, L, d, _dtype_code(q)))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    _check(lib.jetlong_prefill_ie(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"), B, Hq,
                                  Hkv, L, d, int(w0), int(w_pretrained), float(rope_theta),
                                  float(scale), _dtype_code(q), _dev(workspace, "workspace"),
                                  workspace.numel() * workspace.element_size(), _stream(stream)), lib)
    return out


def _host(t, name):
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def prefill_streamed(q_host, k_host, v_host, out_host, q_dev, k_dev, v_dev, out_dev, *, w0: int,
                     w_pretrained: int, rope_theta: float, scale: float | None = None, nchunks: int = 16,
                     stream=None):
    """Prefill from (page-locked) host tensors into ``out_host`` with the transfers
    overlapped with the compute, chunk by chunk; ``*_dev`` are device tensors of
    the same shapes used as staging.  Asynchronous on ``stream``."""
    B, Hq, L, d = q_host.shape
    Hkv = k_host.shape[1]
    for t, n in ((q_dev, "q_dev"), (out_dev, "out_dev"), (out_host, "out_host")):
        if t.shape != q_host.shape or t.dtype != q_host.dtype:
            raise ValueError(f"{n} must match q_host's shape and dtype")
    for t, n in ((k_dev, "k_dev"), (v_dev, "v_dev"), (v_host, "v_host")):
        if t.shape != k_host.shape or t.dtype != k_host.dtype:
            raise ValueError(f"{n} must match k_host's shape and dtype")
    if k_host.shape[0] != B or k_host.shape[2] != L or k_host.shape[3] != d:
        raise ValueError("k_host must be [B, Hkv, L, d] matching q_host")
    _same_dtype((q_host, "q_host"), (k_host, "k_host"))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    lib = load_library()
    _check(lib.jetlong_prefill_streamed(_host(q_host, "q_host"), _host(k_host, "k_host"),
                                        _host(v_host, "v_host"), _host(out_host, "out_host"),
                                        _dev(q_dev, "q_dev"), _dev(k_dev, "k_dev"), _dev(v_dev, "v_dev"),
                                        _dev(out_dev, "out_dev"), B, Hq, Hkv, L, d, int(w0),
                                        int(w_pretrained), float(rope_theta), float(scale),
                                        _dtype_code(q_host), int(nchunks), _stream(stream)), lib)
    return out_host


def prefill_varlen(q, k, v, lens, out=None, *, w0: int, w_pretrained: int, rope_theta: float,
                   scale: float | None = None, with_lse: bool = False, stream=None):
    """Variable-length batch in padded tensors q/out [B,Hq,Lmax,d], k/v
    [B,Hkv,Lmax,d]; sequence b uses rows [0, lens[b]) and its own G.  With
    ``with_lse`` also returns the per-row natural-log LSE [B,Hq,Lmax] (fp32;
    rows past a sequence's length are left as allocated)."""
    import numpy as _np
    import torch
    B, Hq, Lmax, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, Lmax, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, Lmax, d] matching q")
    _same_dtype((q, "q"), (k, "k"), (v, "v"))
    lens = _np.ascontiguousarray(_np.asarray(lens, dtype=_np.int32).reshape(-1))
    if lens.shape[0] != B:
        raise ValueError("lens must have one length per sequence")
    if out is None:
        out = torch.empty_like(q)
    _like(out, q, "out", "q")
    lse = torch.empty((B, Hq, Lmax), dtype=torch.float32, device=q.device) if with_lse else None
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    lib = load_library()
    _check(lib.jetlong_prefill_varlen(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"),
                                      lse.data_ptr() if lse is not None else None, B, Hq, Hkv,
                                      lens.ctypes.data, Lmax, d, int(w0), int(w_pretrained),
                                      float(rope_theta), float(scale), _dtype_code(q),
                                      _stream(stream)), lib)
    return (out, lse) if with_lse else out


def _decode_shapes(q, kcache, vcache):
    if q.dim() != 3 or kcache.dim() != 4:
        raise ValueError("q must be [B, Hq, d] and the caches [B, Hkv, Lcap, d]")
    if vcache.shape != kcache.shape:
        raise ValueError("kcache and vcache must have the same shape")
    if kcache.shape[0] != q.shape[0] or kcache.shape[3] != q.shape[2]:
        raise ValueError("the caches must be [B, Hkv, Lcap, d] with q's B and d")
    _same_dtype((q, "q"), (kcache, "kcache"), (vcache, "vcache"))


def decode_workspace_size(B: int, Hq: int, Hkv: int, Lcap: int, d: int) -> int:
    return int(load_library().jetlong_decode_workspace_size(B, Hq, Hkv, Lcap, d))


def decode_rope_cache(q, kcache, vcache, L: int, out=None, *, w0: int, w_pretrained: int,
                      rope_theta: float, scale: float | None = None, workspace=None, stream=None):
    """One decode step over a standard RoPE cache (key row j stored rotated to
    position j): jetlong_decode_rope_cache."""
    return decode(q, kcache, vcache, L, out, w0=w0, w_pretrained=w_pretrained,
                  rope_theta=rope_theta, scale=scale, workspace=workspace, stream=stream,
                  _entry="jetlong_decode_rope_cache")


def decode(q, kcache, vcache, L: int, out=None, *, w0: int, w_pretrained: int,
           rope_theta: float, scale: float | None = None, workspace=None, stream=None,
           _entry: str = "jetlong_decode"):
    """One decode step: raw q [B,Hq,d] at position L-1 over cache rows [0, L)."""
    import torch
    _decode_shapes(q, kcache, vcache)
    B, Hq, d = q.shape
    _, Hkv, Lcap, _ = kcache.shape
    if out is None:
        out = torch.empty_like(q)
    _like(out, q, "out", "q")
    need = decode_workspace_size(B, Hq, Hkv, Lcap, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    lib = load_library()
    _check(getattr(lib, _entry)(_dev(q, "q"), _dev(kcache, "kcache"), _dev(vcache, "vcache"),
                              _dev(out, "out"), B, Hq, Hkv, int(L), Lcap, d, int(w0),
                              int(w_pretrained), float(rope_theta), float(scale),
                              _dtype_code(q), _dev(workspace, "workspace"),
                              workspace.numel() * workspace.element_size(), _stream(stream)), lib)
    return out


# Size of the library's fixed decode scratch array (JETLONG_DECODE_NOALLOC_SCRATCH_BYTES).
DECODE_NOALLOC_SCRATCH_BYTES = 4 << 20


def decode_noalloc(q, kcache, vcache, L: int, out=None, *, w0: int, w_pretrained: int,
                   rope_theta: float, scale: float | None = None, stream=None):
    """Decode step for callers that cannot allocate device memory.

    Same result as ``decode`` but without a workspace: the library keeps the
    split partials in its own fixed device array (shared by all calls on a
    device, so calls that overlap on the GPU race).  ``out`` should be
    preallocated by such callers; problems too large for the array raise
    JetLongError(INVALID_ARG).
    """
    import torch
    _decode_shapes(q, kcache, vcache)
    B, Hq, d = q.shape
    _, Hkv, Lcap, _ = kcache.shape
    if out is None:
        out = torch.empty_like(q)
    _like(out, q, "out", "q")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    lib = load_library()
    _check(lib.jetlong_decode_noalloc(_dev(q, "q"), _dev(kcache, "kcache"), _dev(vcache, "vcache"),
                                      _dev(out, "out"), B, Hq, Hkv, int(L), Lcap, d, int(w0),
                                      int(w_pretrained), float(rope_theta), float(scale),
                                      _dtype_code(q), _stream(stream)), lib)
    return out


# ---------------------------------------------------------------- paged cache
# kcache, vcache [num_pages, Hkv, page_size, d]; block_table int32 [B, max_pages];
# lens int32 [B] committed rows per request.  All arrays live on the device, so a
# step (block_tables, cache_append, decode_paged or decode_tree, tree_commit) can
# be captured into a CUDA graph.

#
# The host side of a call is as long as a small call itself, so it asks for little:
# torch is looked up once, devices and streams by the raw queries (the public ones
# build objects), each tensor for its type, shape, device and layout.
_torch = None


def _current():
    """(current device, its current stream's handle)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    if not _torch.cuda.is_initialized():
        return -2, None  # then no tensor is on a device either: the argument checks say so
    dev = _torch._C._cuda_getDevice()
    return dev, _torch._C._cuda_getCurrentRawStream(dev)


def _ptr(t, name, dev):
    """Device pointer of a contiguous tensor on device ``dev`` (checks as ``_dev``)."""
    if t.get_device() != dev or not t.is_contiguous():
        return _dev(t, name)
    return t.data_ptr()


def _ints(t, name, shape, dev):
    """Device pointer of an int32 array of the given shape (None stays None)."""
    if t is None:
        return None
    if t.dtype is not _torch.int32 or t.shape != shape:
        raise ValueError(f"{name} must be an int32 tensor of shape {tuple(shape)} (got {t.dtype}, {tuple(t.shape)})")
    if t.get_device() != dev or not t.is_contiguous():
        return _dev(t, name)
    return t.data_ptr()


def _need(t, name):
    if t is None:
        raise ValueError(f"{name} is required")
    return t


def _on(stream):
    """Context in which a call's own tensors are made: those of another stream than the
    current one are allocated on it, so that their memory is free there before the call
    and is not handed out elsewhere until the call is done with it."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    return torch.cuda.stream(stream)


def _caches(kcache, vcache):
    if kcache.dim() != 4 or vcache.shape != kcache.shape:
        raise ValueError("kcache and vcache must both be [num_pages, Hkv, page_size, d]")
    _same_dtype((kcache, "kcache"), (vcache, "vcache"))
    return kcache.shape


class BlockTables(NamedTuple):
    """Result of ``block_tables`` (int32 CUDA tensors; the block table and the free list are updated in place)."""
    lens: "object"        # [B] committed rows (0 for released requests)
    held: "object"        # [B] pages held
    free_count: "object"  # [1] free pages left
    slot_map: "object"    # [n_rows] slot of every new row, -1: none
    row_start: "object"   # [B + 1] first token row of each request
    status: "object"      # [B] 0 granted, 1 no free pages, 2 longer than its table row (both: left out by the other calls), 3 out of range


def block_tables(lens, grow, block_table, held, free_list, free_count, *, page_size: int, num_pages: int, n_rows: int,
                 release=None, lens_out=None, held_out=None, free_count_out=None, slot_map=None, row_start=None,
                 status=None, stream=None) -> BlockTables:
    """Make room for grow[b] new rows of every request and map them to slots
    (jetlong_block_tables).  ``block_table`` [B, max_pages] and ``free_list`` are
    updated in place; the ``*_out`` arrays may be their inputs.  A refused request's
    table gets NO_PAGE where its new rows would be, by which the other calls leave it
    out; a place with lens[b] < 0 and grow[b] == 0 is idle."""
    import torch
    if block_table.dim() != 2 or free_list.dim() != 1:
        raise ValueError("block_table must be [B, max_pages] and free_list one-dimensional")
    B, max_pages = block_table.shape
    made = (lens_out, held_out, free_count_out, slot_map, row_start, status)
    sizes = [n if x is None else 0 for x, n in zip(made, (B, B, 1, n_rows, B + 1, B))]
    if any(sizes) or slot_map is None:
        with _on(stream):  # one allocation for all that the caller did not bring
            new = torch.empty(sum(sizes), dtype=torch.int32, device=block_table.device).split(sizes)
        lens_out, held_out, free_count_out, slot_map, row_start, status = \
            [y if x is None else x for x, y in zip(made, new)]
    lib = _lib or load_library()
    cur, raw = _current()
    reqs, one = (B,), (1,)
    _check(lib.jetlong_block_tables(
        _ints(_need(lens, "lens"), "lens", reqs, cur), _ints(_need(grow, "grow"), "grow", reqs, cur),
        _ints(release, "release", reqs, cur), _ints(_need(held, "held"), "held", reqs, cur),
        _ints(_need(free_count, "free_count"), "free_count", one, cur), _ints(block_table, "block_table", (B, max_pages), cur),
        _ints(free_list, "free_list", free_list.shape, cur), _ints(lens_out, "lens_out", reqs, cur),
        _ints(held_out, "held_out", reqs, cur), _ints(free_count_out, "free_count_out", one, cur),
        _ints(slot_map, "slot_map", (n_rows,), cur), _ints(row_start, "row_start", (B + 1,), cur),
        _ints(status, "status", reqs, cur), B, max_pages, int(page_size), int(num_pages), free_list.shape[0], int(n_rows),
        raw if stream is None else stream.cuda_stream), lib)
    return BlockTables(lens_out, held_out, free_count_out, slot_map, row_start, status)


def _rows(t, name, like, N, dev):
    """Pointer and (token, head) strides of a [N, Hkv, d] tensor whose rows are contiguous."""
    _, Hkv, _, d = like.shape
    if t.shape != (N, Hkv, d) or t.dtype is not like.dtype:
        raise ValueError(f"{name} must be [N, Hkv, d] = {(N, Hkv, d)} with the cache's dtype (got {tuple(t.shape)}, {t.dtype})")
    if t.get_device() != dev:
        _dev(t, name)
    token, head, last = t.stride()
    if last != 1 and N > 0:
        raise ValueError(f"{name} must have contiguous rows (stride 1 in d)")
    # the stride of a dimension of size one is arbitrary and unused
    return t.data_ptr(), token if N > 1 else 0, head if Hkv > 1 else 0


def cache_append(k, v, slot_map, kcache, vcache, stream=None):
    """Write raw rows k, v [N, Hkv, d] (any token and head strides) to their
    slots of the paged cache; slot -1 leaves a row out (jetlong_cache_append)."""
    num_pages, Hkv, page_size, d = _caches(kcache, vcache)
    N = k.shape[0]
    lib = _lib or load_library()
    cur, raw = _current()
    kp, kt, kh = _rows(k, "k", kcache, N, cur)
    vp, vt, vh = _rows(v, "v", kcache, N, cur)
    _check(lib.jetlong_cache_append(kp, vp, _ints(_need(slot_map, "slot_map"), "slot_map", (N,), cur),
                                    _ptr(kcache, "kcache", cur), _ptr(vcache, "vcache", cur), N, Hkv, d, kt, kh, vt, vh,
                                    num_pages, page_size, _dtype_code(kcache),
                                    raw if stream is None else stream.cuda_stream), lib)


def decode_tree_workspace_size(B: int, Hq: int, Hkv: int, d: int, max_nodes: int = 1) -> int:
    return int(load_library().jetlong_decode_tree_workspace_size(B, Hq, Hkv, d, max_nodes))


def _paged_shapes(q, kcache, vcache, block_table):
    num_pages, Hkv, page_size, d = _caches(kcache, vcache)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q must be [N, Hq, d] with the cache's d")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    _same_dtype((q, "q"), (kcache, "kcache"), (vcache, "vcache"))
    return num_pages, Hkv, page_size, d


def decode_paged(q, kcache, vcache, block_table, lens, out=None, *, w0: int, w_pretrained: int, rope_theta: float,
                 scale: float | None = None, workspace=None, stream=None):
    """One decode step of every request over the paged cache: raw q [B, Hq, d],
    request b's query (and its own row) at position lens[b]; requests with
    lens[b] < 0 are idle and their rows of ``out`` untouched (jetlong_decode_paged)."""
    return decode_tree(q, kcache, vcache, block_table, lens, None, None, out, max_nodes=1, w0=w0,
                       w_pretrained=w_pretrained, rope_theta=rope_theta, scale=scale, workspace=workspace,
                       stream=stream)


def decode_tree(q, kcache, vcache, block_table, lens, row_start, parents=None, out=None, *, max_nodes: int, w0: int,
                w_pretrained: int, rope_theta: float, scale: float | None = None, workspace=None, stream=None):
    """Decode a tree of drafted rows per request: raw q [N, Hq, d], request b's
    nodes in token rows [row_start[b], row_start[b + 1]), parents [N] within each
    request (-1: the last committed row; None: chains), node t appended as row
    lens[b] + t (jetlong_decode_tree).  Rows of ``out`` of requests without nodes and
    of refused ones are left as they were.  The kernel follows max_nodes, not the
    nodes of the call: what it holds per unit (at 64 nodes of 4 heads 256 query rows)
    costs time also where only a few of them are used."""
    import torch
    num_pages, Hkv, page_size, d = _paged_shapes(q, kcache, vcache, block_table)
    N, Hq, _ = q.shape
    B, max_pages = block_table.shape
    if row_start is None and N != B:
        raise ValueError("without row_start, q must have one row per request")
    lib = _lib or load_library()
    with _on(stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            workspace = torch.empty(decode_tree_workspace_size(B, Hq, Hkv, d, int(max_nodes)), dtype=torch.uint8,
                                    device=q.device)
    _like(out, q, "out", "q")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    cur, raw = _current()
    _check(lib.jetlong_decode_tree(
        _ptr(q, "q", cur), _ptr(kcache, "kcache", cur), _ptr(vcache, "vcache", cur), _ptr(out, "out", cur),
        _ints(block_table, "block_table", (B, max_pages), cur), _ints(_need(lens, "lens"), "lens", (B,), cur),
        _ints(row_start, "row_start", (B + 1,), cur), _ints(parents, "parents", (N,), cur), B, N, Hq, Hkv, d, num_pages,
        page_size, max_pages, int(max_nodes), int(w0), int(w_pretrained), float(rope_theta), float(scale), _dtype_code(q),
        _ptr(workspace, "workspace", cur), workspace.numel() * workspace.element_size(),
        raw if stream is None else stream.cuda_stream), lib)
    return out


def tree_commit(kcache, vcache, block_table, lens, row_start, parents, last, *, max_nodes: int, lens_out=None,
                n_accepted=None, stream=None):
    """Commit the path to node last[b] (-1: none) of every request: its rows
    become rows lens[b], lens[b] + 1, ... and lens_out = lens + their number; refused
    and idle ones stay as they are (jetlong_tree_commit).  Returns (lens_out, n_accepted)."""
    import torch
    num_pages, Hkv, page_size, d = _caches(kcache, vcache)
    if block_table.dim() != 2 or row_start.dim() != 1:
        raise ValueError("block_table must be [B, max_pages] and row_start [B + 1]")
    B, max_pages = block_table.shape
    with _on(stream):
        lens_out = torch.empty_like(lens) if lens_out is None else lens_out
        n_accepted = torch.empty_like(lens) if n_accepted is None else n_accepted
    # without parents (chains) the token rows are not read and need no bound
    N = 2147483647 if parents is None else parents.numel()
    lib = _lib or load_library()
    cur, raw = _current()
    _check(lib.jetlong_tree_commit(
        _ptr(kcache, "kcache", cur), _ptr(vcache, "vcache", cur), _ints(block_table, "block_table", (B, max_pages), cur),
        _ints(lens, "lens", (B,), cur), _ints(_need(row_start, "row_start"), "row_start", (B + 1,), cur),
        _ints(parents, "parents", (N,), cur), _ints(_need(last, "last"), "last", (B,), cur),
        _ints(lens_out, "lens_out", (B,), cur), _ints(n_accepted, "n_accepted", (B,), cur), B, N, Hkv, d, num_pages,
        page_size, max_pages, int(max_nodes), _dtype_code(kcache), raw if stream is None else stream.cuda_stream), lib)
    return lens_out, n_accepted


def selftest_wait_timeout(stream=None):
    """Launch the bounded-wait self test; the next device_status() raises TIMEOUT."""
    lib = load_library()
    _check(lib.jetlong_selftest_wait_timeout(_stream(stream)), lib)


# Sites of the failure-detection test hook (JETLONG_INJECT_*).
INJECT_PREFILL_KEY_TILE = 1
INJECT_DECODE_COPY = 2


def debug_inject_timeout(site: int, wait_cycles: int):
    """Arm the one-shot test hook: the next prefill or decode call of this thread
    withholds one barrier arrival (``site``) with every bounded wait limited to
    ``wait_cycles`` SM cycles, so its waits expire and the following
    device_status() raises TIMEOUT (jetlong_debug_inject_timeout)."""
    lib = load_library()
    _check(lib.jetlong_debug_inject_timeout(int(site), int(wait_cycles)), lib)


def debug_rope_phase(pos, d: int, rope_theta: float, accurate: bool, stream=None):
    """(cos, sin) of pos[i] * theta_m as the kernels form them: float32 CUDA
    tensor [n, d/2, 2] (test hook jetlong_debug_rope_phase).  pos: int32 CUDA
    tensor holding uint32 positions."""
    import torch
    if pos.dtype != torch.int32:
        raise TypeError("pos must be int32 (uint32 bit patterns)")
    out = torch.empty((pos.numel(), d // 2, 2), dtype=torch.float32, device=pos.device)
    lib = load_library()
    _check(lib.jetlong_debug_rope_phase(_dev(pos, "pos"), pos.numel(), int(d), float(rope_theta),
                                        1 if accurate else 0, _dev(out, "out"), _stream(stream)), lib)
    return out


def debug_tile_plan(P: int, C: int, w0: int, max_kb: int, stream=None):
    """The prefill's tile plan (nR, kE0, nkb) per query block and the class of
    every tile (0 remote, 1 local, 2 both; -1 past nkb): test hook
    jetlong_debug_tile_plan.  Returns (plan [nqb, 3] int32, cls [nqb, max_kb] int8)."""
    import torch
    nqb = (C + 127) // 128
    plan = torch.empty((nqb, 3), dtype=torch.int32, device="cuda")
    cls = torch.full((nqb, max_kb), -1, dtype=torch.int8, device="cuda")
    lib = load_library()
    _check(lib.jetlong_debug_tile_plan(int(P), int(C), int(w0), int(max_kb), _dev(plan, "plan"), _dev(cls, "cls"),
                                       _stream(stream)), lib)
    return plan, cls


def debug_ex2(y, stream=None):
    """2^y as the one-CTA prefill's softmax forms part of its exponentials on the
    FMA pipe (test hook jetlong_debug_ex2).  y: float32 CUDA tensor with an even
    number of elements; returns a tensor of the same shape."""
    import torch
    if y.dtype != torch.float32 or y.numel() % 2:
        raise TypeError("y must be float32 with an even number of elements")
    y = y.contiguous()
    out = torch.empty_like(y)
    lib = load_library()
    _check(lib.jetlong_debug_ex2(_dev(y, "y"), y.numel(), _dev(out, "out"), _stream(stream)), lib)
    return out


def debug_rope_keys(k, G: int, rope_theta: float, remote: bool = True, stream=None):
    """The bf16 prefill's key rotation pass on its own (test hook
    jetlong_debug_rope_keys): k, a bf16 CUDA tensor [planes, L, d], rotated to
    positions j and floor(j / G) times the prefill's key scale 2^e.  Returns
    (kl, kr or None, e); kl and kr are fp16 tensors of k's shape."""
    import ctypes as ct
    import torch
    if k.dtype != torch.bfloat16 or k.dim() != 3:
        raise TypeError("k must be a bf16 tensor [planes, L, d]")
    k = k.contiguous()
    kl = torch.empty(k.shape, dtype=torch.float16, device=k.device)
    kr = torch.empty_like(kl) if remote else None
    ex = ct.c_int(0)
    lib = load_library()
    _check(lib.jetlong_debug_rope_keys(_dev(k, "k"), k.shape[0], k.shape[1], k.shape[2], int(G), float(rope_theta),
                                       _dev(kl, "kl"), _dev(kr, "kr") if remote else None, ct.byref(ex),
                                       _stream(stream)), lib)
    return kl, kr, int(ex.value)


def device_status(stream=None):
    """Synchronise the stream and raise if a kernel's bounded wait expired."""
    lib = load_library()
    _check(lib.jetlong_device_status(_stream(stream)), lib)
