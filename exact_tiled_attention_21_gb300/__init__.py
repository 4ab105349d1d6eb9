"""Exact tiled attention on GB300 (sm_103a) — Python binding of the C ABI.

The functions ``fa_fwd``, ``fa_bwd`` (and its steps ``fa_bwd_preprocess``,
``fa_bwd_dkdv``, ``fa_bwd_dq``), ``fa_decode``, ``fa_bwd_workspace_bytes``,
``fa_decode_workspace_bytes``, ``fa_get_last_device_error``,
``fa_set_wait_timeout_ns``, ``fa_status_string`` and ``fa_version`` carry the
names and arguments of ``include/fa.h`` and only marshal arguments: every step
of the computation runs in the CUDA kernels of ``libfa_gb300.so``.  PyTorch
supplies device memory (``data_ptr``) and the stream.  ``forward``,
``backward`` and ``decode`` are conveniences that allocate the outputs and the
workspace with torch and then call the same entry points.  So are those of the
serving cache held in 8 bits, ``rope``, ``cache_append_fp8``,
``decode_paged_fp8`` and ``cache_evict_fp8``, through a compiled binding
(``csrc/fa_torch.cpp``, ``_fa_torch.so``), since their small calls take less time
on the GPU than ctypes does on the host.  Only ``rope`` takes part in autograd;
the others return results that record no gradient (``backward`` is called for
it).

There is no fallback: if the shared library is missing, or a call returns an
error status, a ``FAError`` is raised.
"""
import ctypes
import math
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "fa.h")

FA_OK = 0
FA_ERR_INVALID_ARG = -1
FA_ERR_UNSUPPORTED = -2
FA_ERR_ALIGNMENT = -3
FA_ERR_WORKSPACE = -4
FA_ERR_CUDA = -5
FA_ERR_TIMEOUT = -6

_lib = None

_NAMES = {FA_OK: "FA_OK", FA_ERR_INVALID_ARG: "FA_ERR_INVALID_ARG",
          FA_ERR_UNSUPPORTED: "FA_ERR_UNSUPPORTED", FA_ERR_ALIGNMENT: "FA_ERR_ALIGNMENT",
          FA_ERR_WORKSPACE: "FA_ERR_WORKSPACE", FA_ERR_CUDA: "FA_ERR_CUDA",
          FA_ERR_TIMEOUT: "FA_ERR_TIMEOUT"}


class FAError(RuntimeError):
    """A C-ABI call returned a status other than FA_OK (or the library is missing)."""

    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (what, _NAMES.get(status, "?"), status))


def build(force=False):
    """Compile libfa_gb300.so in-tree (nvcc, sm_103a) and return its path."""
    from . import _build
    return _build.build(force=force)


def load():
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FAError(FA_ERR_CUDA, "loading %s (not built; call build())" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_bwd_workspace_bytes.restype = sz
    lib.fa_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_fused_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_bwd_fused_workspace_bytes.restype = sz
    lib.fa_bwd_fused.argtypes = [vp] * 9 + [i, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_bwd_fused.restype = i
    lib.fa_bwd_preprocess.argtypes = [vp, vp, vp, i, i, i, i, vp]
    lib.fa_bwd_preprocess.restype = i
    lib.fa_bwd_dkdv.argtypes = [vp] * 8 + [i, i, i, i, i, f, i, vp]
    lib.fa_bwd_dkdv.restype = i
    lib.fa_bwd_dkdv_pair.argtypes = [vp] * 8 + [i, i, i, i, i, f, i, vp]
    lib.fa_bwd_dkdv_pair.restype = i
    lib.fa_bwd_dq.argtypes = [vp] * 7 + [i, i, i, i, i, f, i, vp]
    lib.fa_bwd_dq.restype = i
    lib.fa_decode_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_decode_workspace_bytes.restype = sz
    lib.fa_decode.argtypes = [vp] * 5 + [i, i, i, i, f, i, vp, sz, vp]
    lib.fa_decode.restype = i
    lib.fa_get_last_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    lib.fa_get_last_device_error.restype = i
    lib.fa_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.fa_set_wait_timeout_ns.restype = ctypes.c_uint64
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = i
    lib.fa_fwd_tile_rows.argtypes = [i] * 6
    lib.fa_fwd_tile_rows.restype = i
    lib.fa_work_schedule.argtypes = [i, i, i, i, ctypes.POINTER(ctypes.c_int)]
    lib.fa_work_schedule.restype = i
    ll = ctypes.c_longlong
    lib.fa_rope_table.argtypes = [ctypes.POINTER(ctypes.c_double), i, ctypes.POINTER(ctypes.c_uint64)]
    lib.fa_rope_table.restype = i
    lib.fa_rope.argtypes = [vp, vp] + [ll] * 6 + [vp, vp] + [i] * 6 + [f, i, vp]
    lib.fa_rope.restype = i
    lib.fa_cache_append_fp8.argtypes = [vp, vp] + [ll] * 6 + [vp] * 9 + [i] * 6 + [f] + [i] * 4 + [vp]
    lib.fa_cache_append_fp8.restype = i
    lib.fa_decode_paged_fp8_workspace_bytes.argtypes = [i] * 7
    lib.fa_decode_paged_fp8_workspace_bytes.restype = sz
    lib.fa_decode_paged_fp8.argtypes = [vp] * 10 + [i] * 9 + [f, vp, sz, vp]
    lib.fa_decode_paged_fp8.restype = i
    lib.fa_cache_evict_fp8.argtypes = [vp] * 11 + [i] * 10 + [vp]
    lib.fa_cache_evict_fp8.restype = i
    _lib = lib
    return lib


def declared_symbols():
    """Names of the functions declared in include/fa.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"\b(fa_[a-z_0-9]+)\s*\(", text)))


# ------------------------------------------------------------------ raw entry points
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _raise(status, what):
    if status != FA_OK:
        raise FAError(status, what)


def fa_status_string(status):
    try:
        return load().fa_status_string(int(status)).decode()
    except FAError:
        return "status %d" % status


def fa_version():
    return load().fa_version()


def fa_set_wait_timeout_ns(ns):
    return int(load().fa_set_wait_timeout_ns(int(ns)))


def fa_get_last_device_error(stream=None):
    """Synchronise the stream; return (status, [code, site, block, aux]) and clear the word."""
    detail = (ctypes.c_int * 4)()
    st = load().fa_get_last_device_error(_stream(stream), detail)
    return st, list(detail)


def fa_decode_paged_workspace_bytes(B, Hq, d, num_splits):
    fn = load().fa_decode_paged_workspace_bytes
    fn.argtypes = [ctypes.c_int] * 4
    fn.restype = ctypes.c_size_t
    return int(fn(B, Hq, d, num_splits))


def fa_decode_paged(q, k_pages, v_pages, block_table, seq_lens, o, lse, B, Hq, Hkv, page_size,
                    max_pages, num_pages, d, scale, num_splits, workspace, workspace_bytes, stream=None):
    fn = load().fa_decode_paged
    if fn.argtypes is None:
        vp, i = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 7 + [i] * 7 + [ctypes.c_float, i, vp, ctypes.c_size_t, vp]
        fn.restype = ctypes.c_int
    _raise(fn(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seq_lens), _ptr(o), _ptr(lse),
              B, Hq, Hkv, page_size, max_pages, num_pages, d, float(scale), int(num_splits),
              _ptr(workspace), int(workspace_bytes), _stream(stream)), "fa_decode_paged")


def decode_paged(q, k_pages, v_pages, block_table, seq_lens, scale=None, num_splits=0, stream=None):
    """O [B,Hq,d] bf16 and LSE [B,Hq] fp32 against a paged cache (int32 table and lengths on the device).
    num_splits <= 0: the library's choice."""
    B, Hq, d = q.shape
    num_pages, Hkv, page_size = k_pages.shape[:3]
    max_pages = block_table.shape[1]
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise ValueError("%s must be a contiguous bf16 CUDA tensor" % n)
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_table and seq_lens must be int32")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    ws = torch.empty(fa_decode_paged_workspace_bytes(B, Hq, d, num_splits), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    fa_decode_paged(q, k_pages, v_pages, block_table, seq_lens, o, lse, B, Hq, Hkv, page_size, max_pages,
                    num_pages, d, scale, num_splits, ws, ws.numel(), stream)
    return o, lse


def fa_fwd_window(q, k, v, o, lse, B, H, Nq, Nk, d, scale, window, stream=None):
    fn = load().fa_fwd_window
    if fn.argtypes is None:
        vp, i = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 5 + [i] * 5 + [ctypes.c_float, i, vp]
        fn.restype = i
    _raise(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d, float(scale), int(window),
              _stream(stream)), "fa_fwd_window")


def fa_bwd_window(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, window, workspace,
                  workspace_bytes, stream=None):
    fn = load().fa_bwd_window
    if fn.argtypes is None:
        vp, i = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 9 + [i] * 5 + [ctypes.c_float, i, vp, ctypes.c_size_t, vp]
        fn.restype = i
    _raise(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), B, H, Nq,
              Nk, d, float(scale), int(window), _ptr(workspace), int(workspace_bytes), _stream(stream)),
           "fa_bwd_window")


def fa_fwd_varlen(q, k, v, o, lse, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream=None):
    fn = load().fa_fwd_varlen
    if fn.argtypes is None:
        vp, i = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 7 + [i] * 5 + [ctypes.c_float, i, vp]
        fn.restype = i
    _raise(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(seqlens_q), _ptr(seqlens_k), B, H, Nq, Nk, d,
              float(scale), int(causal), _stream(stream)), "fa_fwd_varlen")


def fa_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal,
                  workspace, workspace_bytes, stream=None):
    fn = load().fa_bwd_varlen
    if fn.argtypes is None:
        vp, i = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 11 + [i] * 5 + [ctypes.c_float, i, vp, ctypes.c_size_t, vp]
        fn.restype = i
    _raise(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv),
              _ptr(seqlens_q), _ptr(seqlens_k), B, H, Nq, Nk, d, float(scale), int(causal), _ptr(workspace),
              workspace_bytes, _stream(stream)), "fa_bwd_varlen")


def fa_fwd_fp8_workspace_bytes(B, H, Nk, d):
    fn = load().fa_fwd_fp8_workspace_bytes
    if fn.argtypes is None:
        fn.argtypes = [ctypes.c_int] * 4
        fn.restype = ctypes.c_size_t
    return fn(B, H, Nk, d)


def fa_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B, H, Nq, Nk, d, scale, causal, workspace,
               workspace_bytes, stream=None):
    fn = load().fa_fwd_fp8
    if fn.argtypes is None:
        vp, i = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 8 + [i] * 5 + [ctypes.c_float, i, vp, ctypes.c_size_t, vp]
        fn.restype = i
    _raise(fn(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), _ptr(o), _ptr(lse),
              B, H, Nq, Nk, d, float(scale), int(causal), _ptr(workspace), workspace_bytes, _stream(stream)),
           "fa_fwd_fp8")


def forward_fp8(q8, k8, v8, q_scale, k_scale, v_scale, scale=None, causal=False, stream=None, workspace=None):
    """O (bf16) and LSE for e4m3 q8 [B,H,Nq,128], k8/v8 [B,H,Nk,128] (uint8 CUDA tensors) with fp32
    scales: q_scale [B*H, ceil(Nq/128)], k_scale [B*H, ceil(Nk/128)], v_scale [B*H]."""
    B, H, Nq, d = q8.shape
    Nk = k8.shape[2]
    for t, n, shp in ((q8, "q8", (B, H, Nq, d)), (k8, "k8", (B, H, Nk, d)), (v8, "v8", (B, H, Nk, d))):
        if not (t.is_cuda and t.dtype == torch.uint8 and t.is_contiguous() and tuple(t.shape) == shp):
            raise ValueError("%s must be a contiguous uint8 CUDA tensor of shape %s" % (n, shp))
    for t, n, shp in ((q_scale, "q_scale", (B * H, -(-Nq // 128))), (k_scale, "k_scale", (B * H, -(-Nk // 128))),
                      (v_scale, "v_scale", (B * H,))):
        if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and tuple(t.shape) == shp):
            raise ValueError("%s must be a contiguous float32 CUDA tensor of shape %s" % (n, shp))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nbytes = fa_fwd_fp8_workspace_bytes(B, H, Nk, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q8.device)
    o = torch.empty((B, H, Nq, d), dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q8.device)
    fa_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B, H, Nq, Nk, d, scale, causal, workspace,
               workspace.numel() * workspace.element_size(), stream)
    return o, lse


def fa_selftest_wait_timeout(timeout_ns, stream=None):
    """Launch the watchdog self-test kernel (a wait that must run out)."""
    fn = load().fa_selftest_wait_timeout
    if fn.argtypes is None:
        fn.argtypes = [ctypes.c_uint64, ctypes.c_void_p]
        fn.restype = ctypes.c_int
    _raise(fn(int(timeout_ns), _stream(stream)), "fa_selftest_wait_timeout")


def fa_bwd_workspace_bytes(B, H, Nq, Nk, d):
    return int(load().fa_bwd_workspace_bytes(B, H, Nq, Nk, d))


def fa_decode_workspace_bytes(B, H, Nk, d, num_splits=0):
    return int(load().fa_decode_workspace_bytes(B, H, Nk, d, num_splits))


def fa_fwd(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, stream=None):
    _raise(load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                         float(scale), int(bool(causal)), _stream(stream)), "fa_fwd")


def fa_work_schedule(n_items, chunk_items, grid, per_chunk):
    """The CTA that takes each work item in the persistent grids' static
    schedule (a list of n_items ints)."""
    owner = (ctypes.c_int * max(1, n_items))()
    _raise(load().fa_work_schedule(n_items, chunk_items, grid, int(bool(per_chunk)), owner), "fa_work_schedule")
    return list(owner)[:n_items]


def fa_fwd_tile_rows(B, H, Nq, Nk, d, causal):
    """Query rows per work tile fa_fwd takes for these sizes (256, or 128 for
    split-KV tiles)."""
    rows = load().fa_fwd_tile_rows(B, H, Nq, Nk, d, int(bool(causal)))
    if rows < 0:
        raise FAError(rows, "fa_fwd_tile_rows")
    return rows


def fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, workspace,
           workspace_bytes, stream=None):
    _raise(load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                         _ptr(dk), _ptr(dv), B, H, Nq, Nk, d, float(scale), int(bool(causal)),
                         _ptr(workspace), int(workspace_bytes), _stream(stream)), "fa_bwd")


def fa_bwd_fused_workspace_bytes(B, H, Nq, Nk, d):
    return load().fa_bwd_fused_workspace_bytes(B, H, Nq, Nk, d)


def fa_bwd_fused(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, workspace,
                 workspace_bytes, stream=None):
    """fa_bwd in one pass over the key tiles (dQ by fp32 reduce-adds; d = 128)."""
    _raise(load().fa_bwd_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                               _ptr(dv), B, H, Nq, Nk, d, float(scale), int(causal), _ptr(workspace),
                               int(workspace_bytes), _stream(stream)), "fa_bwd_fused")


def fa_bwd_preprocess(o, dO, delta, B, H, Nq, d, stream=None):
    _raise(load().fa_bwd_preprocess(_ptr(o), _ptr(dO), _ptr(delta), B, H, Nq, d, _stream(stream)),
           "fa_bwd_preprocess")


def fa_bwd_dkdv(q, k, v, lse, delta, dO, dk, dv, B, H, Nq, Nk, d, scale, causal, stream=None):
    _raise(load().fa_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(delta), _ptr(dO), _ptr(dk),
                              _ptr(dv), B, H, Nq, Nk, d, float(scale), int(bool(causal)),
                              _stream(stream)), "fa_bwd_dkdv")


def fa_bwd_dkdv_pair(q, k, v, lse, delta, dO, dk, dv, B, H, Nq, Nk, d, scale, causal, stream=None):
    """fa_bwd_dkdv on CTA pairs (cta_group::2 products; d = 128)."""
    _raise(load().fa_bwd_dkdv_pair(_ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(delta), _ptr(dO), _ptr(dk),
                                   _ptr(dv), B, H, Nq, Nk, d, float(scale), int(causal), _stream(stream)),
           "fa_bwd_dkdv_pair")


def fa_bwd_dq(q, k, v, lse, delta, dO, dq, B, H, Nq, Nk, d, scale, causal, stream=None):
    _raise(load().fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(delta), _ptr(dO), _ptr(dq),
                            B, H, Nq, Nk, d, float(scale), int(bool(causal)), _stream(stream)),
           "fa_bwd_dq")


def fa_decode(q, kcache, vcache, o, lse, B, H, Nk, d, scale, num_splits, workspace,
              workspace_bytes, stream=None):
    _raise(load().fa_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(o), _ptr(lse), B, H, Nk,
                            d, float(scale), int(num_splits), _ptr(workspace),
                            int(workspace_bytes), _stream(stream)), "fa_decode")


def fa_decode_noalloc(q, kcache, vcache, o, lse, B, H, Nk, d, scale, num_splits, stream=None):
    """fa_decode without a workspace: the partials go to the library's fixed
    scratch array (for callers that may not allocate; see include/fa.h)."""
    fn = load().fa_decode_noalloc
    if fn.argtypes is None:
        vp, i = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 5 + [i, i, i, i, ctypes.c_float, i, vp]
        fn.restype = ctypes.c_int
    _raise(fn(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(o), _ptr(lse), B, H, Nk, d, float(scale),
              int(num_splits), _stream(stream)), "fa_decode_noalloc")


def fa_rope_table(inv_freq):
    """Turns per position (Python ints, 2^-64 turn) of the angles per position ``inv_freq`` (radians)."""
    fn = load().fa_rope_table
    n = len(inv_freq)
    turns = (ctypes.c_uint64 * max(1, n))()
    _raise(fn((ctypes.c_double * max(1, n))(*inv_freq), n, turns), "fa_rope_table")
    return list(turns)


def fa_rope(x, y, x_strides, y_strides, positions, turns, B, H, N, d, rot, interleaved, magnitude, inverse,
            stream=None):
    _raise(load().fa_rope(_ptr(x), _ptr(y), *x_strides, *y_strides, _ptr(positions), _ptr(turns), B, H, N, d, rot,
                          int(bool(interleaved)), float(magnitude), int(bool(inverse)), _stream(stream)), "fa_rope")


def fa_cache_append_fp8(k, v, k_strides, v_strides, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens,
                        new_lens, positions, turns, B, Hkv, N, d, rot, interleaved, magnitude, page_size,
                        scale_block, max_pages, num_pages, stream=None):
    _raise(load().fa_cache_append_fp8(_ptr(k), _ptr(v), *k_strides, *v_strides, _ptr(k_pages), _ptr(v_pages),
                                      _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(seq_lens),
                                      _ptr(new_lens), _ptr(positions), _ptr(turns), B, Hkv, N, d, rot,
                                      int(bool(interleaved)), float(magnitude), page_size, scale_block, max_pages,
                                      num_pages, _stream(stream)), "fa_cache_append_fp8")


def fa_decode_paged_fp8_workspace_bytes(B, Hq, Hkv, Nq, d, max_tokens, weights):
    return load().fa_decode_paged_fp8_workspace_bytes(B, Hq, Hkv, Nq, d, max_tokens, int(bool(weights)))


def fa_decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, o, lse, weights, B, Hq, Hkv,
                        Nq, page_size, scale_block, max_pages, num_pages, d, scale, workspace, workspace_bytes,
                        stream=None):
    _raise(load().fa_decode_paged_fp8(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale),
                                      _ptr(block_table), _ptr(seq_lens), _ptr(o), _ptr(lse), _ptr(weights), B, Hq,
                                      Hkv, Nq, page_size, scale_block, max_pages, num_pages, d, float(scale),
                                      _ptr(workspace), int(workspace_bytes), _stream(stream)), "fa_decode_paged_fp8")


def fa_cache_evict_fp8(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, weights, new_table, new_lens,
                       new_weights, kept, B, Hkv, page_size, scale_block, max_pages, new_max_pages, num_pages, d,
                       keep, recent, stream=None):
    _raise(load().fa_cache_evict_fp8(_ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
                                     _ptr(seq_lens), _ptr(weights), _ptr(new_table), _ptr(new_lens),
                                     _ptr(new_weights), _ptr(kept), B, Hkv, page_size, scale_block, max_pages,
                                     new_max_pages, num_pages, d, int(keep), int(recent), _stream(stream)),
           "fa_cache_evict_fp8")


# ------------------------------------------------------------------ conveniences
def _check(t, name, shape):
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
        raise ValueError("%s must be a contiguous bf16 CUDA tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _lens(t, B, name):
    if not (t.is_cuda and t.dtype == torch.int32 and t.is_contiguous() and t.shape == (B,)):
        raise ValueError("%s must be a contiguous int32 CUDA tensor of shape (%d,)" % (name, B))


def forward(q, k, v, scale=None, causal=False, stream=None, seqlens_q=None, seqlens_k=None):
    """O, LSE for q [B,H,Nq,d], k/v [B,H,Nk,d] (bf16 CUDA).  LSE is fp32 [B,H,Nq].

    With seqlens_q / seqlens_k (int32 [B] on the device, both or neither):
    per-sequence lengths within the padded tensors (fa_fwd_varlen)."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    _check(q, "q", (B, H, Nq, d))
    _check(k, "k", (B, H, Nk, d))
    _check(v, "v", (B, H, Nk, d))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if seqlens_q is not None or seqlens_k is not None:
        _lens(seqlens_q, B, "seqlens_q")
        _lens(seqlens_k, B, "seqlens_k")
        fa_fwd_varlen(q, k, v, o, lse, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream)
    else:
        fa_fwd(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, stream)
    return o, lse


def backward(q, k, v, o, lse, dO, scale=None, causal=False, stream=None, workspace=None, seqlens_q=None,
             seqlens_k=None, fused=False):
    """dQ, dK, dV (bf16) for the forward output o / lse and upstream gradient dO.
    fused=True: fa_bwd_fused (one pass, dQ by fp32 reduce-adds; d = 128)."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    for t, n, s in ((q, "q", (B, H, Nq, d)), (k, "k", (B, H, Nk, d)), (v, "v", (B, H, Nk, d)),
                    (o, "o", (B, H, Nq, d)), (dO, "dO", (B, H, Nq, d))):
        _check(t, n, s)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if fused and (seqlens_q is not None or seqlens_k is not None):
        raise ValueError("fused=True takes no sequence lengths")
    nbytes = (fa_bwd_fused_workspace_bytes if fused else fa_bwd_workspace_bytes)(B, H, Nq, Nk, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if seqlens_q is not None or seqlens_k is not None:
        _lens(seqlens_q, B, "seqlens_q")
        _lens(seqlens_k, B, "seqlens_k")
        fa_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal,
                      workspace, workspace.numel() * workspace.element_size(), stream)
    else:
        (fa_bwd_fused if fused else fa_bwd)(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, causal,
                                            workspace, workspace.numel() * workspace.element_size(), stream)
    return dq, dk, dv


def decode(q, kcache, vcache, scale=None, num_splits=0, stream=None, workspace=None,
           want_lse=True):
    """O [B,H,d] bf16 (and LSE [B,H] fp32) for one query per (b, h) against the caches."""
    B, H, d = q.shape
    Nk = kcache.shape[2]
    _check(q, "q", (B, H, d))
    _check(kcache, "kcache", (B, H, Nk, d))
    _check(vcache, "vcache", (B, H, Nk, d))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nbytes = fa_decode_workspace_bytes(B, H, Nk, d, num_splits)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device) if want_lse else None
    fa_decode(q, kcache, vcache, o, lse, B, H, Nk, d, scale, num_splits, workspace,
              workspace.numel() * workspace.element_size(), stream)
    return (o, lse) if want_lse else o


# ------------------------------------------------------------------ rotary positions and the 8-bit cache
_torch_binding = None


def _native():
    """The native binding (csrc/fa_torch.cpp): checks, allocations and the C call in one step."""
    global _torch_binding
    if _torch_binding is None:
        load()
        try:
            from . import _fa_torch
        except ImportError as e:
            raise FAError(FA_ERR_CUDA, "loading _fa_torch.so (not built; call build()): %s" % e)
        _torch_binding = _fa_torch
    return _torch_binding


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on_stream(stream, t):
    """torch's current stream set to ``stream``, so that what a call allocates belongs to the stream that uses it.
    A handle of 0 is the default stream (of which ExternalStream would make a new one)."""
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=t.device) if handle else torch.cuda.default_stream(t.device)
    _need(stream.device == t.device, "stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_context=None, beta_fast=32.0,
                     beta_slow=1.0):
    """Angle per position of each of rot / 2 pairs (Python floats), and the magnitude for ``rope``.

    scaling None: base^(-2i/rot).  "linear": positions divided by factor.  "ntk": the base times
    factor^(rot / (rot - 2)), which stretches the longest wave by factor and leaves the shortest.  "yarn": by parts;
    pairs that turn more than beta_fast times within original_context tokens keep their frequency, those that turn
    less than beta_slow times are divided by factor, the ones between are blended linearly in their number of turns;
    magnitude 0.1 ln(factor) + 1.  A model that was trained with other frequencies (such as a blend that is linear in
    the pair's index between two rounded bounds) takes its own: any list goes to ``rope_table``.
    """
    _need(rot >= 2 and rot % 2 == 0, "rot must be even and at least 2")
    _need(base > 0 and factor >= 1.0, "base must be positive and factor at least 1")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling is None or scaling == "ntk":
        return f, 1.0
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    _need(scaling == "yarn", "scaling must be None, 'linear', 'ntk' or 'yarn'")
    _need(original_context is not None and original_context >= 1, "yarn needs the original context's length")
    _need(beta_fast > beta_slow, "beta_fast must be above beta_slow")
    out = []
    for x in f:
        keep = (original_context * x / (2.0 * math.pi) - beta_slow) / (beta_fast - beta_slow)
        keep = min(1.0, max(0.0, keep))
        out.append(x * keep + x / factor * (1.0 - keep))
    return out, 0.1 * math.log(factor) + 1.0


def rope_table(inv_freq, device="cuda"):
    """The device table (int64 [rot / 2], the bits of fa_rope_table's values) of angles per position in radians."""
    turns = fa_rope_table([float(x) for x in inv_freq])
    return torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device=device)


class _Rope(torch.autograd.Function):
    """rope where a gradient is recorded: the gradient is the rotation by the opposite angles."""

    @staticmethod
    def forward(ctx, x, turns, positions, interleaved, magnitude, inverse):
        ctx.save_for_backward(turns, positions)
        ctx.form = interleaved, magnitude, inverse
        return rope(x, turns, positions, interleaved, magnitude, inverse)

    @staticmethod
    def backward(ctx, g):
        turns, positions = ctx.saved_tensors
        interleaved, magnitude, inverse = ctx.form
        if g.stride(3) != 1 or g.data_ptr() % 16 or any(s % 8 for s in g.stride()[:3]):
            g = g.clone(memory_format=torch.contiguous_format)  # rows that the kernel does not take
        return (rope(g, turns, positions, interleaved, magnitude, not inverse),) + (None,) * 5


def rope(x, turns, positions=None, interleaved=False, magnitude=1.0, inverse=False, out=None, stream=None):
    """x [B,H,N,d] (bf16, any strides that fa_rope takes) rotated by its tokens' positions: pairs 0 .. len(turns) - 1,
    the columns behind them copied.  turns: rope_table(...).  positions: int32 [B,N] on the device, or None (0..N-1).
    inverse=True turns back: the gradient of x from the gradient of the result.  out: where to write (may be x, but not
    overlap it otherwise); default a new contiguous tensor.  Where x requires a gradient, the result records it (out
    must then be None)."""
    if stream is not None:
        with _on_stream(stream, x):
            return rope(x, turns, positions, interleaved, magnitude, inverse, out)
    if (getattr(x, "requires_grad", False) or getattr(out, "requires_grad", False)) and torch.is_grad_enabled():
        _need(out is None, "out does not record a gradient: call under torch.no_grad(), or without out")
        return _Rope.apply(x, turns, positions, interleaved, magnitude, inverse)
    r = (_torch_binding or _native()).rope(x, turns, positions, interleaved, magnitude, inverse, out)
    if r.__class__ is int:
        raise FAError(r, "fa_rope")
    return r


def cache_append_fp8(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, new_lens=None, turns=None,
                     positions=None, interleaved=False, magnitude=1.0, stream=None):
    """Writes k, v [B,Hkv,N,d] (bf16, any strides that fa_rope takes) behind the seq_lens[b] tokens that the paged
    8-bit cache holds of each sequence: the first new_lens[b] of them (None: all N).  With turns, k is rotated on the
    way (positions int32 [B,N], or None: seq_lens[b] + i).  Changes the pages and scales, not seq_lens."""
    if stream is not None:
        with _on_stream(stream, k):
            return cache_append_fp8(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, new_lens, turns,
                                    positions, interleaved, magnitude)
    st = (_torch_binding or _native()).append(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, new_lens,
                                              turns, positions, interleaved, magnitude)
    if st != FA_OK:
        raise FAError(st, "fa_cache_append_fp8")


def decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, scale=None, weights=None,
                     stream=None, workspace=None):
    """O [B,Hq,Nq,d] bf16 and LSE [B,Hq,Nq] fp32 of the last Nq tokens (q [B,Hq,Nq,d], or [B,Hq,d] for one, which
    gives O [B,Hq,d] and LSE [B,Hq]) over the paged 8-bit cache, which holds them already.  weights: fp32
    [B,Hkv,max_pages*page] to which every token's attention weight is added, or None; with them the workspace holds a
    score per query row and slot of the table, so the table should be no wider than the longest sequence needs."""
    if stream is not None:
        with _on_stream(stream, q):
            return decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, scale, weights,
                                    None, workspace)
    r = (_torch_binding or _native()).decode(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, scale,
                                             weights, workspace)
    if r.__class__ is int:
        raise FAError(r, "fa_decode_paged_fp8")
    return r


def cache_evict_fp8(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, weights, new_table, keep, recent=0,
                    stream=None):
    """Copies, of each sequence and kv head, the last ``recent`` tokens and the keep - recent others of largest
    accumulated weight into the pages of new_table (int32 [B, new_max_pages], disjoint from the pages read).  Returns
    (new_lens int32 [B], new_weights fp32 and kept int32 [B,Hkv,new_max_pages*page]): the kept tokens' weights and
    source indices, 0 and -1 behind them."""
    if stream is not None:
        with _on_stream(stream, k_pages):
            return cache_evict_fp8(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, weights, new_table, keep,
                                   recent)
    r = (_torch_binding or _native()).evict(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, weights,
                                            new_table, keep, recent)
    if r.__class__ is int:
        raise FAError(r, "fa_cache_evict_fp8")
    return r
