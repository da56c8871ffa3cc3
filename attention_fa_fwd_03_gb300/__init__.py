"""Exact scaled-dot-product attention on GB300 (sm_103a), for training and for serving from a paged cache.

Thin Python binding over the C ABI of ``libfa_gb300.so`` (declared in
``include/fa.h``): it only turns torch tensors into pointers and sizes, calls
the C function, and raises ``FaError`` on a non-zero status. Every step of the
computation runs in the library's CUDA kernels; there is no fallback. If the
library has not been built, every call raises. The paged-cache calls, made once
per layer and token, go through a compiled binding (csrc/paged_binding.cpp)
instead of ctypes.

    import attention_fa_fwd_03_gb300 as fa
    fa.fa_fwd(q, k, v, o, lse, scale, causal=True)
    ws = torch.empty(fa.fa_bwd_workspace_size(B, Hq, Tq), dtype=torch.uint8, device="cuda")
    fa.fa_bwd(q, k, v, o, do, lse, dq, dk, dv, scale, causal=True, workspace=ws)

Serving from a paged key/value cache (a pool of pages and a page table):

    kv = fa.PagedKV(k_pool, v_pool, page_table, kv_lens, k_bounds=bounds)   # kept from step to step
    kv_lens += 1                                                            # the new token counts
    fa.fa_kv_append(kv, k, v, cos=cos, sin=sin, q=q, q_out=qr)              # rotate, append
    fa.fa_paged_fwd(kv, qr, o, lse, scale, causal=True, workspace=ws)       # attention over the cache
    fa.fa_page_select(kv, qr, sel, sel_lens, keep_last=2, workspace=ws2)    # or over chosen pages:
    fa.fa_paged_fwd(kv, qr, o, lse, scale, causal=True, sel=sel, sel_lens=sel_lens, workspace=ws)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

__all__ = ["FA_FP16", "FA_BF16", "FaError", "fa_fwd", "fa_bwd", "fa_bwd_preprocess", "fa_bwd_dkv",
           "fa_bwd_dq", "fa_bwd_workspace_size",
           "PagedKV", "fa_kv_append", "fa_paged_fwd", "fa_paged_workspace_size", "fa_page_select",
           "fa_page_select_workspace_size",
           "fa_status_string", "fa_device_status", "fa_abi_version", "fa_selftest_wait_timeout",
           "fa_set_wait_limit_cycles", "library", "library_path"]

FA_FP16 = 0
FA_BF16 = 1
STATUS_NAMES = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED_HEAD_DIM",
                3: "FA_ERR_UNSUPPORTED_DTYPE", 4: "FA_ERR_MISALIGNED", 5: "FA_ERR_LAUNCH",
                6: "FA_ERR_TIMEOUT", 7: "FA_ERR_BAD_INDEX"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


class _PagedKVStruct(ctypes.Structure):
    """fa_paged_kv of include/fa.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_bounds", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("dt", ctypes.c_int)]


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({_status_text(status)})")


def library_path() -> str:
    return os.path.join(_HERE, "libfa_gb300.so")


def library():
    """The loaded C library (ctypes), with argument types declared."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library not built: {path} is missing "
                               "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
        lib = ctypes.CDLL(path)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i, vp]
        lib.fa_fwd.restype = i
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i,
                               vp, sz, vp]
        lib.fa_bwd.restype = i
        lib.fa_bwd_preprocess.argtypes = [vp, vp, vp, i, i, i, i, i, vp]
        lib.fa_bwd_preprocess.restype = i
        lib.fa_bwd_dkv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i,
                                   vp]
        lib.fa_bwd_dkv.restype = i
        lib.fa_bwd_dq.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i, vp]
        lib.fa_bwd_dq.restype = i
        lib.fa_bwd_workspace_size.argtypes = [i, i, i]
        lib.fa_bwd_workspace_size.restype = sz
        kvp, i64p = ctypes.POINTER(_PagedKVStruct), ctypes.c_void_p
        lib.fa_kv_append.argtypes = [kvp, vp, i64p, vp, i64p, vp, i64p, vp, i, i, vp, vp, vp, i, i,
                                     i, vp]
        lib.fa_kv_append.restype = i
        lib.fa_paged_fwd.argtypes = [kvp, vp, vp, vp, i, i, f, i, i, vp, vp, vp, i, vp, sz, vp]
        lib.fa_paged_fwd.restype = i
        lib.fa_paged_workspace_size.argtypes = [i, i, i, i]
        lib.fa_paged_workspace_size.restype = sz
        lib.fa_page_select.argtypes = [kvp, vp, i, i, i, i, vp, vp, vp, sz, vp]
        lib.fa_page_select.restype = i
        lib.fa_page_select_workspace_size.argtypes = [i, i, i]
        lib.fa_page_select_workspace_size.restype = sz
        lib.fa_status_string.argtypes = [i]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i, vp]
        lib.fa_device_status.restype = i
        lib.fa_abi_version.argtypes = []
        lib.fa_abi_version.restype = i
        lib.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
        lib.fa_selftest_wait_timeout.restype = i
        lib.fa_set_wait_limit_cycles.argtypes = [ctypes.c_ulonglong]
        lib.fa_set_wait_limit_cycles.restype = i
        _lib = lib
        return lib


def _status_text(st: int) -> str:
    try:
        return library().fa_status_string(st).decode()
    except Exception:  # library missing while formatting an error
        return "?"


def _check(st: int, what: str) -> None:
    if st != 0:
        raise FaError(st, what)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return FA_FP16
    if t.dtype == torch.bfloat16:
        return FA_BF16
    raise FaError(3, f"dtype {t.dtype}")


def _ptr(t) -> int:
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous (row-major [B, H, T, D])")
    return t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def fa_abi_version() -> int:
    return library().fa_abi_version()


def fa_status_string(st: int) -> str:
    return library().fa_status_string(st).decode()


def fa_bwd_workspace_size(B: int, Hq: int, Tq: int) -> int:
    return int(library().fa_bwd_workspace_size(B, Hq, Tq))


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool = False, window: int = 0,
           stream=None) -> None:
    """O and LSE for q [B,Hq,Tq,D], k/v [B,Hkv,Tkv,D] (fp16 or bf16, contiguous,
    on the GPU); o [B,Hq,Tq,D] same dtype, lse [B,Hq,Tq] fp32 are written."""
    B, Hq, Tq, D = q.shape
    Hkv, Tkv = k.shape[1], k.shape[2]
    st = library().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Tq, Tkv, D,
                          float(scale), int(bool(causal)), int(window), _dtype_code(q),
                          _stream(stream))
    _check(st, "fa_fwd")


def fa_bwd(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool = False,
           window: int = 0, workspace=None, stream=None) -> None:
    """dQ, dK, dV for the forward that produced o and lse. ``workspace`` is a
    device tensor of at least fa_bwd_workspace_size(B, Hq, Tq) bytes."""
    B, Hq, Tq, D = q.shape
    Hkv, Tkv = k.shape[1], k.shape[2]
    if workspace is None:
        raise ValueError("fa_bwd needs a workspace tensor (the library never allocates)")
    nbytes = workspace.numel() * workspace.element_size()
    st = library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                          _ptr(dk), _ptr(dv), B, Hq, Hkv, Tq, Tkv, D, float(scale),
                          int(bool(causal)), int(window), _dtype_code(q), _ptr(workspace),
                          nbytes, _stream(stream))
    _check(st, "fa_bwd")


def _ws_ptr(workspace) -> int:
    if workspace is None:
        raise ValueError("a D-vector workspace tensor is required (the library never allocates)")
    return _ptr(workspace)


def fa_bwd_preprocess(o, do, workspace, stream=None) -> None:
    """D-vector rowsum(dO * O) into ``workspace`` (fp32 [B, Hq, Tq])."""
    B, Hq, Tq, D = o.shape
    st = library().fa_bwd_preprocess(_ptr(o), _ptr(do), _ws_ptr(workspace), B, Hq, Tq, D,
                                     _dtype_code(o), _stream(stream))
    _check(st, "fa_bwd_preprocess")


def fa_bwd_dkv(q, k, v, do, lse, workspace, dk, dv, scale: float, causal: bool = False,
               window: int = 0, stream=None) -> None:
    """dK, dV given the D-vector already in ``workspace``."""
    B, Hq, Tq, D = q.shape
    Hkv, Tkv = k.shape[1], k.shape[2]
    st = library().fa_bwd_dkv(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(lse), _ws_ptr(workspace),
                              _ptr(dk), _ptr(dv), B, Hq, Hkv, Tq, Tkv, D, float(scale),
                              int(bool(causal)), int(window), _dtype_code(q), _stream(stream))
    _check(st, "fa_bwd_dkv")


def fa_bwd_dq(q, k, v, do, lse, workspace, dq, scale: float, causal: bool = False,
              window: int = 0, stream=None) -> None:
    """dQ given the D-vector already in ``workspace``."""
    B, Hq, Tq, D = q.shape
    Hkv, Tkv = k.shape[1], k.shape[2]
    st = library().fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(lse), _ws_ptr(workspace),
                             _ptr(dq), B, Hq, Hkv, Tq, Tkv, D, float(scale), int(bool(causal)),
                             int(window), _dtype_code(q), _stream(stream))
    _check(st, "fa_bwd_dq")


# ------------------------------------------------------------- paged cache
class PagedKV:
    """A paged key/value cache as the paged calls take it: the pools and the
    tables that say which pages each sequence has (see include/fa.h).

    ``k`` and ``v`` [num_pages, Hkv, page_size, D] fp16 or bf16, page_size 16 to
    256; ``page_table`` [B, max_pages] and ``kv_lens`` [B] int32; ``k_bounds``
    [num_pages, Hkv, 2, D] or None. All contiguous on one CUDA device. The
    object keeps the tensors alive and is made once: page_table and kv_lens are
    read by every call and updated in place by the caller. Its attributes cannot
    be assigned (``kv.kv_lens += 1`` updates in place): calls go to the tensors
    it was made with.
    """

    __slots__ = ("k", "v", "page_table", "kv_lens", "k_bounds", "device", "dtype", "B", "Hkv", "D",
                 "num_pages", "page_size", "max_pages", "_handle", "_calls")

    def __init__(self, k, v, page_table, kv_lens, k_bounds=None):
        import torch
        if k.dim() != 4 or page_table.dim() != 2:
            raise ValueError("k and v are [num_pages, Hkv, page_size, D], page_table is [B, max_pages]")
        put = functools.partial(object.__setattr__, self)
        for name, value in zip(("num_pages", "Hkv", "page_size", "D", "B", "max_pages", "device", "dtype"),
                               (*k.shape, *page_table.shape, k.device, k.dtype)):
            put(name, value)
        code = _dtype_code(k)
        ptrs = [_ptr(k), self._pointer("v", v, k.shape, k.dtype),
                0 if k_bounds is None else
                self._pointer("k_bounds", k_bounds, (self.num_pages, self.Hkv, 2, self.D), k.dtype),
                self._pointer("page_table", page_table, page_table.shape, torch.int32),
                self._pointer("kv_lens", kv_lens, (self.B,), torch.int32)]
        if max(self.num_pages, self.Hkv, self.page_size, self.D, self.B, self.max_pages) > 2 ** 31 - 1:
            raise ValueError("a size is beyond 32 bits")
        calls = _paged_calls()
        for name, value in (("k", k), ("v", v), ("k_bounds", k_bounds), ("page_table", page_table), ("kv_lens", kv_lens),
                            ("_calls", calls),
                            ("_handle", calls.handle(*ptrs, self.B, self.Hkv, self.D, self.num_pages, self.page_size,
                                                     self.max_pages, code, self.device.index))):
            put(name, value)

    def __setattr__(self, name: str, value) -> None:
        if value is getattr(self, name, self):
            return  # `kv.kv_lens += 1` has updated the tensor and assigns it again
        raise AttributeError(f"PagedKV.{name} cannot be assigned: update the tensor in place or make a new PagedKV")

    def __delattr__(self, name: str) -> None:
        raise AttributeError(f"PagedKV.{name} cannot be deleted")

    def _pointer(self, name: str, t, shape, dtype) -> int:
        if t.dtype != dtype or t.shape != shape:
            raise ValueError(f"{name}: expected {dtype} of shape {list(shape)}, got {t.dtype} of shape {list(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{name}: expected on {self.device}, got {t.device}")
        return _ptr(t)


def _paged_calls():
    """The compiled binding of the paged calls."""
    library()
    try:
        from . import _paged
    except ImportError as e:
        raise RuntimeError("binding of the paged calls not built for this PyTorch: _paged.so is missing or does not load "
                           f"(run `python -c 'import __graft_entry__ as g; g.build()'`): {e}") from e
    return _paged


def fa_kv_append(kv: PagedKV, k, v, cos=None, sin=None, interleaved: bool = False, q=None,
                 q_out=None, new_lens=None, stream=None) -> None:
    """Append T new tokens per sequence to the cache: keys rotated by their
    position, values copied, page bounds updated where the cache keeps them.

    ``k`` and ``v`` [B, Hkv, T, D] and ``q`` [B, Hq, T, D] may be any views
    with a contiguous innermost index and other strides in multiples of 8, such
    as transposed slices of a fused projection. The rotated queries go to
    ``q_out`` (contiguous). ``cos`` and ``sin`` [positions, rot_dim / 2] fp32, or
    None for no rotation. ``kv.kv_lens`` counts the new tokens already;
    ``new_lens`` [B] int32 says how many of the T rows of each sequence are
    tokens (None: all)."""
    st = kv._calls.kv_append(kv._handle, k, v, cos, sin, interleaved, q, q_out, new_lens, stream)
    if st != 0:
        raise FaError(st, "fa_kv_append")


def fa_paged_workspace_size(Hq: int, Hkv: int, Tq: int, D: int) -> int:
    return int(library().fa_paged_workspace_size(Hq, Hkv, Tq, D))


def fa_paged_fwd(kv: PagedKV, q, o, lse, scale: float, causal: bool = False, window: int = 0,
                 new_lens=None, sel=None, sel_lens=None, workspace=None, stream=None) -> None:
    """O and LSE of Tq <= 8 new tokens per sequence over the paged cache.

    ``q`` and ``o`` [B, Hq, Tq, D], ``lse`` [B, Hq, Tq] fp32, contiguous. The new
    tokens are the last keys of the cache (``kv.kv_lens`` counts them); causal
    and window masks go by position in the sequence. ``sel`` [B, Hkv, n_sel]
    and ``sel_lens`` [B, Hkv] int32 restrict each KV head to these pages.
    ``workspace`` has fa_paged_workspace_size(Hq, Hkv, Tq, D) bytes."""
    st = kv._calls.paged_fwd(kv._handle, q, o, lse, scale, causal, window, new_lens, sel, sel_lens,
                             workspace, stream)
    if st != 0:
        raise FaError(st, "fa_paged_fwd")


def fa_page_select_workspace_size(B: int, Hkv: int, max_pages: int) -> int:
    return int(library().fa_page_select_workspace_size(B, Hkv, max_pages))


def fa_page_select(kv: PagedKV, q, sel, sel_lens, keep_first: int = 0, keep_last: int = 1,
                   workspace=None, stream=None) -> None:
    """The pages that attention of one new token reads, chosen per sequence and
    KV head by the bounds of their keys (``kv.k_bounds``): ``sel`` [B, Hkv,
    n_sel] int32 gets the page numbers in ascending order, then -1, and
    ``sel_lens`` [B, Hkv] int32 how many. ``q`` [B, Hq, 1, D]. The first
    ``keep_first`` and last ``keep_last`` pages are always chosen.
    ``workspace`` has fa_page_select_workspace_size(B, Hkv, max_pages) bytes."""
    st = kv._calls.page_select(kv._handle, q, sel, sel_lens, keep_first, keep_last, workspace, stream)
    if st != 0:
        raise FaError(st, "fa_page_select")


def fa_selftest_wait_timeout(timeout_ms: int, stream=None) -> None:
    """Launch the library's bounded-wait self-test (see include/fa.h): a wait
    that can never complete gives up after ``timeout_ms``; read the result
    with fa_device_status()."""
    _check(library().fa_selftest_wait_timeout(int(timeout_ms), _stream(stream)),
           "fa_selftest_wait_timeout")


def fa_set_wait_limit_cycles(cycles: int) -> None:
    """Bound (SM clock cycles) of the kernels' ordinary waits for every later
    launch in this process; 0 restores the default. A diagnostic for tests of
    the give-up path (see include/fa.h)."""
    _check(library().fa_set_wait_limit_cycles(int(cycles)), "fa_set_wait_limit_cycles")


def fa_device_status(clear: bool = True, stream=None) -> int:
    """Synchronise ``stream`` and return the device status word (0 = no bounded
    wait gave up). Raises nothing; the caller inspects the bits."""
    bits = ctypes.c_uint(0)
    library().fa_device_status(ctypes.byref(bits), int(bool(clear)), _stream(stream))
    return int(bits.value)
