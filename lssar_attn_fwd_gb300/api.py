"""ctypes binding of liblssar_attn_fwd.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module
only checks tensor metadata, takes raw device pointers and the current CUDA
stream from PyTorch and calls the C ABI declared in
``include/lssar_attn_fwd.h``.  There is no fallback: if the library is not
built, or a call fails, an exception is raised.
"""

import ctypes
import os
import struct

from .inputs import MODE_LSSA, MODE_LSSAR, MODE_SIGMOID_RW, MODE_SOFTMAX, MODE_SOFTMAX_RW  # noqa: F401

_LIB = None

_EXPORTS = (
    "lssar_attn_fwd",
    "lssar_attn_fwd_simt",
    "lssar_attn_fwd_profiled",
    "lssar_attn_fwd_noalloc",
    "lssar_attn_fwd_heads_p",
    "lssar_attn_decode",
    "lssar_attn_fwd_train",
    "lssar_attn_bwd",
    "lssar_attn_bwd_simt",
    "lssar_attn_fwd_train_heads_p",
    "lssar_attn_bwd_heads_p",
    "lssar_selftest_stall",
    "lssar_schedule_plan",
    "lssar_decode_plan",
    "lssar_paged_append",
    "lssar_paged_decode",
    "lssar_paged_evict",
    "lssar_status_string",
    "lssar_device_error_word",
    "lssar_abi_version",
)


DTYPE_BF16 = 0
DTYPE_FP16 = 1


class PagedCacheDesc(ctypes.Structure):
    """lssar_paged_cache_t of the C ABI."""

    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("page_stride", ctypes.c_longlong), ("n_pages", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("B", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("d", ctypes.c_int), ("dtype", ctypes.c_int)]


class LssarError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"lssar status {status}: {message}")
        self.status = status


def lib_path(debug=False):
    name = "liblssar_attn_fwd_debug.so" if debug else "liblssar_attn_fwd.so"
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", name)


_DEBUG_LIB = None


def load_debug_library():
    """Loads the debug-check build of the library (built with
    ``build(debug=True)``): the same C ABI, with device-side bounds checks
    that record codes 101-105 in its own device error word.  The functions of
    this module keep calling the default library; call the debug one through
    the returned handle (the argument declarations are the same)."""
    global _DEBUG_LIB
    if _DEBUG_LIB is None:
        _DEBUG_LIB = _open(lib_path(debug=True))
    return _DEBUG_LIB


def load_library():
    """Loads the shared library (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        _LIB = _open(lib_path())
    return _LIB


def _open(path):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m lssar_attn_fwd_gb300.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    fwd_args = [ctypes.c_void_p] * 4 + [ctypes.c_int] * 6 + [ctypes.c_void_p]
    for name in ("lssar_attn_fwd", "lssar_attn_fwd_simt", "lssar_attn_fwd_noalloc", "lssar_attn_decode"):
        fn = getattr(lib, name)
        fn.argtypes = fwd_args
        fn.restype = ctypes.c_int
    lib.lssar_attn_fwd_heads_p.argtypes = ([ctypes.c_void_p] * 4 + [ctypes.c_int] * 4 +
                                           [ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.c_void_p])
    lib.lssar_attn_fwd_heads_p.restype = ctypes.c_int
    lib.lssar_attn_fwd_train.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_int] * 6 + [ctypes.c_void_p]
    lib.lssar_attn_fwd_train.restype = ctypes.c_int
    lib.lssar_attn_fwd_train_heads_p.argtypes = ([ctypes.c_void_p] * 5 + [ctypes.c_int] * 4 +
                                                 [ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.c_void_p])
    lib.lssar_attn_fwd_train_heads_p.restype = ctypes.c_int
    lib.lssar_attn_bwd_heads_p.argtypes = ([ctypes.c_void_p] * 8 + [ctypes.c_int] * 4 +
                                           [ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.c_void_p])
    lib.lssar_attn_bwd_heads_p.restype = ctypes.c_int
    for name in ("lssar_attn_bwd", "lssar_attn_bwd_simt"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.c_void_p] * 8 + [ctypes.c_int] * 6 + [ctypes.c_void_p]
        fn.restype = ctypes.c_int
    lib.lssar_attn_fwd_profiled.argtypes = fwd_args + [ctypes.c_void_p] * 3
    lib.lssar_attn_fwd_profiled.restype = ctypes.c_int
    lib.lssar_schedule_plan.argtypes = [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int)] * 2
    lib.lssar_schedule_plan.restype = ctypes.c_int
    lib.lssar_decode_plan.argtypes = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int)] * 4
    lib.lssar_decode_plan.restype = ctypes.c_int
    # (the cache description and the stride arrays by address: a PagedCacheDesc by
    # reference, or bytes)
    ptr, num = ctypes.c_void_p, ctypes.c_int
    lib.lssar_paged_append.argtypes = [ptr] * 5 + [num] + [ptr] * 6
    lib.lssar_paged_decode.argtypes = [ptr] * 4 + [num] * 3 + [ptr] * 3
    lib.lssar_paged_evict.argtypes = [ptr] * 3 + [num] * 3 + [ptr] * 4
    for name in ("lssar_paged_append", "lssar_paged_decode", "lssar_paged_evict"):
        getattr(lib, name).restype = ctypes.c_int
    lib.lssar_selftest_stall.argtypes = [ctypes.c_void_p]
    lib.lssar_selftest_stall.restype = ctypes.c_int
    lib.lssar_status_string.argtypes = [ctypes.c_int]
    lib.lssar_status_string.restype = ctypes.c_char_p
    lib.lssar_device_error_word.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.lssar_device_error_word.restype = ctypes.c_int
    lib.lssar_abi_version.argtypes = []
    lib.lssar_abi_version.restype = ctypes.c_int
    return lib


def status_string(status):
    return load_library().lssar_status_string(int(status)).decode()


def call_raw(name, q_ptr, k_ptr, v_ptr, out_ptr, B, H, L, d, p, mode, stream_handle):
    """Calls a forward entry point with raw integer pointers; returns the status."""
    fn = getattr(load_library(), name)
    return fn(ctypes.c_void_p(q_ptr), ctypes.c_void_p(k_ptr), ctypes.c_void_p(v_ptr),
              ctypes.c_void_p(out_ptr), int(B), int(H), int(L), int(d), int(p), int(mode),
              ctypes.c_void_p(stream_handle))


def _check(status):
    if status != 0:
        raise LssarError(status, status_string(status))


def _stream_of(stream, device):
    """The torch stream of a ``stream`` argument (a torch stream or a raw handle)."""
    import torch
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)


def _make(stream, device, make):
    """A result tensor that a call on ``stream`` (None: the current one) makes for
    itself.  Its memory comes in the order of the stream that writes it: a block
    freed on the current stream may still be read or written by work queued
    there.  The current stream, which may use the result, is noted for its release."""
    import torch
    if stream is None:
        return make()
    s = _stream_of(stream, device)
    with torch.cuda.stream(s):
        t = make()
    current = torch.cuda.current_stream(device)
    if current != s:
        t.record_stream(current)
    return t


def _forward(name, q, k, v, p, mode, out, stream):
    import torch

    for t in (q, k, v):
        if not isinstance(t, torch.Tensor):
            raise TypeError("q, k, v must be torch tensors")
        if t.device.type != "cuda" or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous bfloat16 CUDA tensors")
        if t.dim() != 4 or t.shape != q.shape:
            raise ValueError("q, k, v must share one [B, H, L, d] shape")
    if k.device != q.device or v.device != q.device:
        raise ValueError("q, k, v must be on one device")
    B, H, L, d = q.shape
    if out is None:
        out = _make(stream, q.device, lambda: torch.empty_like(q))
    elif (out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous()
          or out.device != q.device):
        raise ValueError("out must be a contiguous bfloat16 tensor shaped like q on q's device")
    with torch.cuda.device(q.device):
        if stream is None:
            stream = torch.cuda.current_stream(q.device)
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        _check(call_raw(name, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                        B, H, L, d, p, mode, handle))
    return out


def lssar_attn_fwd(q, k, v, p=3, mode=MODE_LSSAR, out=None, stream=None):
    """Causal LSSAR / LSSA / softmax attention forward on the tensor-core kernel.

    q, k, v: contiguous bf16 CUDA tensors [B, H, L, d] (d = 64 or 128).
    p: re-weighting exponent (modes 2-4).  mode: 0 softmax, 1 LSSA, 2 LSSAR,
    3 re-weighting on a softmax normaliser, 4 sigmoid + L1 + re-weighting.
    Runs asynchronously on ``stream`` (default: the current stream).
    """
    return _forward("lssar_attn_fwd", q, k, v, p, mode, out, stream)


def lssar_attn_fwd_simt(q, k, v, p=3, mode=MODE_LSSAR, out=None, stream=None):
    """Same operation on the plain CUDA-core kernel (cross-check only)."""
    return _forward("lssar_attn_fwd_simt", q, k, v, p, mode, out, stream)


def call_train(q_ptr, k_ptr, v_ptr, out_ptr, stats_ptr, B, H, L, d, p, mode, stream_handle):
    """Raw call of lssar_attn_fwd_train; returns the status."""
    return load_library().lssar_attn_fwd_train(
        *(ctypes.c_void_p(x) for x in (q_ptr, k_ptr, v_ptr, out_ptr, stats_ptr)),
        int(B), int(H), int(L), int(d), int(p), int(mode), ctypes.c_void_p(stream_handle))


def call_bwd(name, ptrs, B, H, L, d, p, mode, stream_handle):
    """Raw call of a backward entry point; ptrs = (q, k, v, dout, stats, dq,
    dk, dv) integer device pointers.  Returns the status."""
    return getattr(load_library(), name)(
        *(ctypes.c_void_p(x) for x in ptrs), int(B), int(H), int(L), int(d), int(p), int(mode),
        ctypes.c_void_p(stream_handle))


def _check_like(q, *ts):
    import torch
    for t in ts:
        if (not isinstance(t, torch.Tensor) or t.shape != q.shape or t.dtype != torch.bfloat16
                or not t.is_contiguous() or t.device != q.device):
            raise ValueError("tensors must be contiguous bfloat16 CUDA tensors shaped like q")


def lssar_attn_fwd_train(q, k, v, p=3, mode=MODE_LSSAR, out=None, stats=None, stream=None):
    """Training forward: returns (out, stats), stats [B, H, L, 4] float32 row
    statistics {m, kappa, beta, W} for :func:`lssar_attn_bwd_simt`."""
    import torch
    if q.device.type != "cuda":
        raise ValueError("q must be a CUDA tensor")
    _check_like(q, q, k, v)
    B, H, L, d = q.shape
    out = _make(stream, q.device, lambda: torch.empty_like(q)) if out is None else out
    _check_like(q, out)
    if stats is None:
        stats = _make(stream, q.device, lambda: torch.empty((B, H, L, 4), dtype=torch.float32, device=q.device))
    elif stats.shape != (B, H, L, 4) or stats.dtype != torch.float32 or not stats.is_contiguous():
        raise ValueError("stats must be a contiguous float32 [B, H, L, 4] tensor")
    with torch.cuda.device(q.device):
        s = torch.cuda.current_stream(q.device) if stream is None else stream
        _check(call_train(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), stats.data_ptr(),
                          B, H, L, d, p, mode, s.cuda_stream))
    return out, stats


def _backward(name, q, k, v, dout, stats, p, mode, stream):
    import torch
    if q.device.type != "cuda":
        raise ValueError("q must be a CUDA tensor")
    _check_like(q, q, k, v, dout)
    B, H, L, d = q.shape
    if stats.shape != (B, H, L, 4) or stats.dtype != torch.float32 or not stats.is_contiguous():
        raise ValueError("stats must be the float32 [B, H, L, 4] tensor of lssar_attn_fwd_train")
    dq, dk, dv = (_make(stream, q.device, lambda: torch.empty_like(q)) for _ in range(3))
    with torch.cuda.device(q.device):
        s = torch.cuda.current_stream(q.device) if stream is None else stream
        ptrs = tuple(t.data_ptr() for t in (q, k, v, dout, stats, dq, dk, dv))
        _check(call_bwd(name, ptrs, B, H, L, d, p, mode, s.cuda_stream))
    return dq, dk, dv


def lssar_attn_bwd(q, k, v, dout, stats, p=3, mode=MODE_LSSAR, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * out) on the tensor-core backward,
    from the row statistics of :func:`lssar_attn_fwd_train` (same q, k, v, p,
    mode).  Runs asynchronously on ``stream`` (default: the current stream)."""
    return _backward("lssar_attn_bwd", q, k, v, dout, stats, p, mode, stream)


def lssar_attn_bwd_simt(q, k, v, dout, stats, p=3, mode=MODE_LSSAR, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * out) on the plain CUDA-core
    backward (cross-check path), from the row statistics of
    :func:`lssar_attn_fwd_train`."""
    return _backward("lssar_attn_bwd_simt", q, k, v, dout, stats, p, mode, stream)


def call_heads_p(q_ptr, k_ptr, v_ptr, out_ptr, B, H, L, d, p_per_head, mode, stream_handle):
    """Raw call of lssar_attn_fwd_heads_p; returns the status."""
    arr = (ctypes.c_int * max(1, len(p_per_head)))(*[int(x) for x in p_per_head])
    ptr = arr if len(p_per_head) else None
    return load_library().lssar_attn_fwd_heads_p(
        ctypes.c_void_p(q_ptr), ctypes.c_void_p(k_ptr), ctypes.c_void_p(v_ptr),
        ctypes.c_void_p(out_ptr), int(B), int(H), int(L), int(d), ptr, int(mode),
        ctypes.c_void_p(stream_handle))


def lssar_attn_fwd_heads_p(q, k, v, p_per_head, mode=MODE_LSSAR, out=None, stream=None):
    """Re-weighting modes with one exponent per head (p_per_head: H ints)."""
    import torch
    B, H, L, d = q.shape
    if len(p_per_head) != H:
        raise ValueError("p_per_head must hold one exponent per head")
    if out is None:
        out = _make(stream, q.device, lambda: torch.empty_like(q))
    with torch.cuda.device(q.device):
        s = torch.cuda.current_stream(q.device) if stream is None else stream
        _check(call_heads_p(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            B, H, L, d, p_per_head, mode, s.cuda_stream))
    return out


def _int_array(values):
    arr = (ctypes.c_int * max(1, len(values)))(*[int(x) for x in values])
    return arr if len(values) else None


def call_train_heads_p(q_ptr, k_ptr, v_ptr, out_ptr, stats_ptr, B, H, L, d, p_per_head, mode, stream_handle):
    """Raw call of lssar_attn_fwd_train_heads_p; returns the status."""
    return load_library().lssar_attn_fwd_train_heads_p(
        *(ctypes.c_void_p(x) for x in (q_ptr, k_ptr, v_ptr, out_ptr, stats_ptr)),
        int(B), int(H), int(L), int(d), _int_array(p_per_head), int(mode), ctypes.c_void_p(stream_handle))


def call_bwd_heads_p(ptrs, B, H, L, d, p_per_head, mode, stream_handle):
    """Raw call of lssar_attn_bwd_heads_p; ptrs as for :func:`call_bwd`."""
    return load_library().lssar_attn_bwd_heads_p(
        *(ctypes.c_void_p(x) for x in ptrs), int(B), int(H), int(L), int(d), _int_array(p_per_head),
        int(mode), ctypes.c_void_p(stream_handle))


def lssar_attn_fwd_train_heads_p(q, k, v, p_per_head, mode=MODE_LSSAR, stream=None):
    """Training forward with one re-weighting exponent per head: returns
    (out, stats) for :func:`lssar_attn_bwd_heads_p` (same p_per_head)."""
    import torch
    if q.device.type != "cuda":
        raise ValueError("q must be a CUDA tensor")
    _check_like(q, q, k, v)
    B, H, L, d = q.shape
    if len(p_per_head) != H:
        raise ValueError("p_per_head must hold one exponent per head")
    out = _make(stream, q.device, lambda: torch.empty_like(q))
    stats = _make(stream, q.device, lambda: torch.empty((B, H, L, 4), dtype=torch.float32, device=q.device))
    with torch.cuda.device(q.device):
        s = torch.cuda.current_stream(q.device) if stream is None else stream
        _check(call_train_heads_p(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), stats.data_ptr(),
                                  B, H, L, d, p_per_head, mode, s.cuda_stream))
    return out, stats


def lssar_attn_bwd_heads_p(q, k, v, dout, stats, p_per_head, mode=MODE_LSSAR, stream=None):
    """Tensor-core backward with one re-weighting exponent per head, from the
    statistics of :func:`lssar_attn_fwd_train_heads_p`."""
    import torch
    if q.device.type != "cuda":
        raise ValueError("q must be a CUDA tensor")
    _check_like(q, q, k, v, dout)
    B, H, L, d = q.shape
    if len(p_per_head) != H:
        raise ValueError("p_per_head must hold one exponent per head")
    if stats.shape != (B, H, L, 4) or stats.dtype != torch.float32 or not stats.is_contiguous():
        raise ValueError("stats must be the float32 [B, H, L, 4] tensor of lssar_attn_fwd_train_heads_p")
    dq, dk, dv = (_make(stream, q.device, lambda: torch.empty_like(q)) for _ in range(3))
    with torch.cuda.device(q.device):
        s = torch.cuda.current_stream(q.device) if stream is None else stream
        ptrs = tuple(t.data_ptr() for t in (q, k, v, dout, stats, dq, dk, dv))
        _check(call_bwd_heads_p(ptrs, B, H, L, d, p_per_head, mode, s.cuda_stream))
    return dq, dk, dv


def lssar_attn_decode(q, k_cache, v_cache, p=3, mode=MODE_LSSAR, out=None, stream=None):
    """One new query row per head (position L) against a K/V cache.

    q: [B, H, d] bf16; k_cache, v_cache: [B, H, L, d] bf16 (contiguous, CUDA).
    Returns out [B, H, d] bf16, equal to row L of the full causal forward.
    """
    import torch
    for t in (q, k_cache, v_cache):
        if t.device.type != "cuda" or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("q, k_cache, v_cache must be contiguous bfloat16 CUDA tensors")
    B, H, L, d = k_cache.shape
    if v_cache.shape != k_cache.shape or tuple(q.shape) != (B, H, d):
        raise ValueError("shapes must be q [B, H, d] and caches [B, H, L, d]")
    if out is None:
        out = _make(stream, q.device, lambda: torch.empty_like(q))
    with torch.cuda.device(q.device):
        s = torch.cuda.current_stream(q.device) if stream is None else stream
        _check(call_raw("lssar_attn_decode", q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                        out.data_ptr(), B, H, L, d, p, mode, s.cuda_stream))
    return out


# lssar_paged_cache_t and stride arrays as bytes: the paged calls are small
# enough that marshalling is a good part of their time (a ctypes structure and
# two arrays cost as much as a launch).
_CACHE = struct.Struct("@PPPPqiiiiiii0q")   # (0q: padded to the structure's size)
_pack_2 = struct.Struct("@2q").pack
_pack_3 = struct.Struct("@3q").pack


def _paged_cache(k_pages, v_pages, table, lens):
    """Checks the tensors of a paged cache; returns (its C description, B, Hkv,
    capacity, d, device index)."""
    import torch
    for t in (k_pages, v_pages, table, lens):
        if not isinstance(t, torch.Tensor):
            raise TypeError("k_pages, v_pages, table and lens must be torch tensors")
    dev = k_pages.get_device() if k_pages.is_cuda else -1
    if dev < 0 or v_pages.get_device() != dev or table.get_device() != dev or lens.get_device() != dev:
        raise ValueError("k_pages, v_pages, table and lens must be CUDA tensors on one device")
    shape, dtype = k_pages.shape, k_pages.dtype
    if len(shape) != 4 or v_pages.shape != shape or v_pages.dtype is not dtype:
        raise ValueError("k_pages and v_pages must share one [n_pages, Hkv, page_size, d] shape and type")
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("k_pages and v_pages must be bfloat16 or float16")
    n_pages, Hkv, ps, d = shape
    if n_pages < 1 or Hkv < 1 or ps < 1:
        raise ValueError("k_pages and v_pages must hold at least one page, head and token")
    kst, vst = k_pages.stride(), v_pages.stride()
    inner = (ps * d, d, 1)
    if (kst[1:] != inner or vst[1:] != inner or kst[0] != vst[0]) and (
            not k_pages[0].is_contiguous() or not v_pages[0].is_contiguous() or (n_pages > 1 and kst[0] != vst[0])):
        raise ValueError("each page must be contiguous, and K and V must share the stride between pages")
    if table.dtype is not torch.int32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous int32 [B, max_pages] tensor")
    B, max_pages = table.shape
    if lens.dtype is not torch.int32 or lens.shape != (B,) or not lens.is_contiguous():
        raise ValueError("lens must be a contiguous int32 [B] tensor")
    # the stride of a single page is never used
    desc = _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(),
                       kst[0] if n_pages > 1 else Hkv * ps * d, n_pages, max_pages, ps, B, Hkv, d,
                       DTYPE_BF16 if dtype is torch.bfloat16 else DTYPE_FP16)
    return desc, B, Hkv, max_pages * ps, d, dev


def _slots(name, t, shape, dtype, dev):
    """The pointer of a [B, Hkv, capacity] tensor of per-slot values, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} [B, Hkv, max_pages * page_size] tensor on the cache's device")
    return t.data_ptr()


def _per_sequence(name, t, B, dev):
    """The pointer of a [B] int32 tensor, or None."""
    import torch
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape != (B,) or not t.is_contiguous() or not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous int32 [B] tensor on the cache's device")
    return t.data_ptr()


def _int32(name, value):
    value = int(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits")
    return value


def _paged_call(name, dev, stream, *args):
    """Calls an entry point on the cache's device and the given (default: the
    current) stream."""
    import torch
    fn = getattr(_LIB or load_library(), name)
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream_of(stream, dev).cuda_stream
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != 0:
        _check(status)


def lssar_paged_append(k_new, v_new, k_pages, v_pages, table, lens, counts=None, first_positions=None, scores=None,
                       positions=None, lens_out=None, stream=None):
    """Puts new tokens' keys and values into the pages of their sequences.

    k_new, v_new: [B, Hkv, n, d] (or [B, Hkv, d] for one token) of the cache's
    type, any strides that are multiples of 8 elements with d contiguous.
    k_pages, v_pages: [n_pages, Hkv, page_size, d] bf16 or fp16 (page_size a
    multiple of 8 up to 256, d = 64 or 128); table: [B, max_pages] int32 page
    numbers; lens: [B] int32 cached tokens.  counts: [B] int32, the first
    counts[b] of the n tokens are appended (default: all).  first_positions:
    [B] int32 position of the first of them (default: lens).  scores (float32)
    and positions (int32), [B, Hkv, max_pages * page_size]: the new slots
    become 0 and the tokens' positions.  Returns the new lengths (lens_out, which
    may not be lens itself).
    Runs asynchronously on ``stream`` (default: the current stream).
    """
    import torch
    desc, B, Hkv, cap, d, dev = _paged_cache(k_pages, v_pages, table, lens)
    if k_new.dim() == 3 and v_new.dim() == 3:
        k_new, v_new = k_new.unsqueeze(2), v_new.unsqueeze(2)
    shape, dtype = k_new.shape, k_pages.dtype
    if (len(shape) != 4 or v_new.shape != shape or k_new.dtype is not dtype or v_new.dtype is not dtype
            or not k_new.is_cuda or not v_new.is_cuda or k_new.get_device() != dev or v_new.get_device() != dev):
        raise ValueError("k_new and v_new must share one [B, Hkv, n, d] shape, with the cache's type and device")
    n = shape[2]
    if (shape[0], shape[1], shape[3]) != (B, Hkv, d):
        raise ValueError("k_new and v_new must be [B, Hkv, n, d] with the cache's B, Hkv and d")
    kst, vst = k_new.stride(), v_new.stride()
    if n and (kst[3] != 1 or vst[3] != 1):
        raise ValueError("the last dimension of k_new and v_new must be contiguous")
    if lens_out is None:
        lens_out = torch.empty_like(lens) if stream is None else _make(stream, dev, lambda: torch.empty_like(lens))
    slots = (B, Hkv, cap)
    _paged_call("lssar_paged_append", dev, stream, desc, k_new.data_ptr(), _pack_3(*kst[:3]), v_new.data_ptr(),
                _pack_3(*vst[:3]), n, _per_sequence("counts", counts, B, dev),
                _per_sequence("first_positions", first_positions, B, dev),
                _slots("scores", scores, slots, torch.float32, dev), _slots("positions", positions, slots, torch.int32, dev),
                _per_sequence("lens_out", lens_out, B, dev))
    return lens_out


def lssar_paged_decode(q, k_pages, v_pages, table, lens, p=3, mode=MODE_LSSAR, scores=None, scores_out=None, out=None,
                       stream=None):
    """One new query row per head against a paged cache, in every mode.

    q: [B, H, d] of the cache's type (d contiguous, other strides multiples of
    8), H a multiple of Hkv, at most 128 * Hkv (query head h reads key head
    h // (H // Hkv)); the cache as in :func:`lssar_paged_append`, the new token
    already appended.  Returns out [B, H, d], row lens[b] of the attention over
    each sequence's cached tokens (zeros for an empty sequence).  scores:
    float32 [B, Hkv, max_pages * page_size]; each cached token's slot of
    scores_out (default: scores itself) becomes scores plus the normalised
    weights that the token gets from the query heads of its key head.
    Runs asynchronously on ``stream`` (default: the current stream).
    """
    import torch
    desc, B, Hkv, cap, d, dev = _paged_cache(k_pages, v_pages, table, lens)
    shape, dtype = q.shape, q.dtype
    if (len(shape) != 3 or shape[0] != B or shape[2] != d or dtype is not k_pages.dtype or not q.is_cuda
            or q.get_device() != dev):
        raise ValueError("q must be [B, H, d] with the cache's B, d, type and device")
    qst = q.stride()
    if qst[2] != 1:
        raise ValueError("the last dimension of q must be contiguous")
    if scores is None and scores_out is not None:
        raise ValueError("scores_out needs scores")
    if scores_out is None:
        scores_out = scores
    if out is None:
        make = lambda: torch.empty(shape, dtype=dtype, device=q.device)   # noqa: E731
        out = make() if stream is None else _make(stream, dev, make)
    elif (out.shape != shape or out.dtype is not dtype or not out.is_contiguous() or not out.is_cuda
          or out.get_device() != dev):
        raise ValueError("out must be a contiguous [B, H, d] tensor of q's type on the cache's device")
    slots = (B, Hkv, cap)
    _paged_call("lssar_paged_decode", dev, stream, desc, q.data_ptr(), _pack_2(*qst[:2]), out.data_ptr(), shape[1],
                _int32("p", p), _int32("mode", mode), _slots("scores", scores, slots, torch.float32, dev),
                _slots("scores_out", scores_out, slots, torch.float32, dev))
    return out


def lssar_paged_evict(k_pages, v_pages, table, lens, scores, positions, keep, recent=0, sinks=0, scores_out=None,
                      positions_out=None, lens_out=None, stream=None):
    """Cuts every sequence with more than ``keep`` cached tokens to ``keep``.

    Per key head the tokens of the highest scores stay (ties: the lower slot),
    and before them the protected ones: position < sinks or position > newest
    position - recent (recent + sinks <= keep).  Kept tokens behind slot
    ``keep`` move into the evicted slots before it, in the pages as in scores
    and positions ([B, Hkv, max_pages * page_size] float32 and int32); with
    scores_out and positions_out (both or neither) these are read only.
    Returns (new lengths, scores_out, positions_out); lens_out may not be lens
    itself.  Runs asynchronously on ``stream`` (default: the current stream).
    """
    import torch
    desc, B, Hkv, cap, d, dev = _paged_cache(k_pages, v_pages, table, lens)
    if (scores_out is None) != (positions_out is None):
        raise ValueError("scores_out and positions_out go together")
    if scores_out is None:
        scores_out, positions_out = scores, positions
    if lens_out is None:
        lens_out = torch.empty_like(lens) if stream is None else _make(stream, dev, lambda: torch.empty_like(lens))
    slots = (B, Hkv, cap)
    _paged_call("lssar_paged_evict", dev, stream, desc, _slots("scores", scores, slots, torch.float32, dev),
                _slots("positions", positions, slots, torch.int32, dev), _int32("keep", keep), _int32("recent", recent),
                _int32("sinks", sinks), _slots("scores_out", scores_out, slots, torch.float32, dev),
                _slots("positions_out", positions_out, slots, torch.int32, dev),
                _per_sequence("lens_out", lens_out, B, dev))
    return lens_out, scores_out, positions_out


def lssar_attn_fwd_profiled(q, k, v, p, mode, out, stream, ev_start, ev_main, ev_end):
    """The tensor-core forward recording caller-owned torch.cuda.Events around
    the prologue and the attention kernel (each event must have been recorded
    once before, so that its CUDA handle exists; None skips that event)."""
    B, H, L, d = q.shape
    handle = lambda e: ctypes.c_void_p(None if e is None else e.cuda_event)  # noqa: E731
    status = load_library().lssar_attn_fwd_profiled(
        ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()), ctypes.c_void_p(v.data_ptr()),
        ctypes.c_void_p(out.data_ptr()), B, H, L, d, int(p), int(mode),
        ctypes.c_void_p(stream.cuda_stream), handle(ev_start), handle(ev_main), handle(ev_end))
    _check(status)
    return out


def decode_plan(B, H, L, d):
    """Launch plan of lssar_attn_decode for these sizes on the current device:
    dict(path=0 cluster | 1 cooperative | 2 three launches, launches,
    chunks, chunk_rows)."""
    vals = [ctypes.c_int(0) for _ in range(4)]
    _check(load_library().lssar_decode_plan(B, H, L, d, *(ctypes.byref(v) for v in vals)))
    return dict(zip(("path", "launches", "chunks", "chunk_rows"), (v.value for v in vals)))


def selftest_stall():
    """Test only: launches a decode step whose copies are withheld, so that its
    bounded waits give up (about 2 s); read the code with device_error_word()."""
    import torch
    _check(load_library().lssar_selftest_stall(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))


def device_error_word():
    """Reads and clears the device error word (synchronises the device)."""
    w = ctypes.c_uint(0)
    _check(load_library().lssar_device_error_word(ctypes.byref(w)))
    return w.value
