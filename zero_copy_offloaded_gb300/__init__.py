"""Zero-copy host-resident KV-cache attention for GB300 (DirectKV's hot path).

A thin ctypes binding over ``libdkv.so`` whose C ABI is ``include/dkv.h``.
Every function here only marshals arguments (tensor -> device pointer,
stream -> cudaStream_t) and calls the library of the same name; every step
of the computation runs in the library's CUDA kernels.  There is no CPU or
PyTorch fallback: if the library is missing or a call fails, a
``DkvError`` is raised.

PyTorch is used only as plumbing for device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import numpy as np

__all__ = [
    "DkvError", "BF16", "FP16", "lib", "lib_path", "KVCache",
    "dkv_cache_alloc", "dkv_free", "dkv_cache_host_ptrs", "dkv_cache_device_ptrs",
    "dkv_cache_set_lengths", "dkv_cache_get_lengths", "dkv_cache_info", "dkv_cache_reserve",
    "dkv_cache_set_tuning", "dkv_decode", "dkv_prefill", "dkv_sync_status", "dkv_status_str",
    "dkv_last_error", "dkv_probe_read", "dkv_probe_write", "dkv_probe_launch", "dkv_attend_naive",
    "dkv_decode_staged", "dkv_prefill_staged", "dkv_prefill_naive", "dkv_decode_unfused", "dkv_last_launch_count", "dkv_cache_kernel_timing",
    "dkv_cache_last_kernel_ms", "dkv_cache_alloc_paged", "dkv_cache_set_page_table",
    "PagedKVCache", "LayeredKVCache", "dkv_cache_alloc_layered", "dkv_decode_layer",
    "dkv_prefill_layer", "dkv_step_graph_capture", "dkv_step_graph_launch",
    "dkv_cache_alloc_ex", "KV_FORMATS", "dkv_decode_noalloc", "dkv_decode_noalloc_status",
    "dkv_decode_noalloc_debug_withhold", "dkv_pci_numa_node", "dkv_numa_probe",
    "dkv_step_plan", "dkv_qkv_append", "dkv_paged_attend", "dkv_paged_attend_workspace",
    "dkv_paged_attend_debug_withhold",
    "dkv_block_append", "dkv_block_attend",
    "dkv_pages_fork", "dkv_pages_compact", "dkv_pages_copy", "dkv_pages_workspace",
    "rope_table", "MAX_STEP_BATCH",
]

BF16 = 0
FP16 = 1
_DTYPE = {"bf16": BF16, "fp16": FP16, BF16: BF16, FP16: FP16}
STATUS = {0: "DKV_OK", 1: "DKV_ERR_INVALID_ARG", 2: "DKV_ERR_UNSUPPORTED", 3: "DKV_ERR_CAPACITY",
          4: "DKV_ERR_NO_MAPPED_MEMORY", 5: "DKV_ERR_ALLOC", 6: "DKV_ERR_CUDA",
          7: "DKV_ERR_TIMEOUT"}

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "_build", "libdkv.so")


class DkvError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{where}: {self.name}: {detail}")


class _CacheInfo(ctypes.Structure):
    _fields_ = [("host_pinned_bytes", ctypes.c_size_t),
                ("device_workspace_bytes", ctypes.c_size_t),
                ("device_staging_bytes", ctypes.c_size_t),
                ("batch", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("dtype", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("max_pages_per_seq", ctypes.c_int),
                ("layers", ctypes.c_int), ("kv_format", ctypes.c_int),
                ("numa_node_wanted", ctypes.c_int), ("numa_node", ctypes.c_int)]


class _CacheDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("dtype", ctypes.c_int), ("kv_format", ctypes.c_int), ("layers", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("max_pages_per_seq", ctypes.c_int)]


# The argument structures of include/dkv.h, packed in one call (native alignment)
_APPEND = struct.Struct("@3P3q10P10i3f")
_ATTEND = struct.Struct("@PqPPPPPPPPN10i2f")
_BLOCK_APPEND = struct.Struct("@3P3q12P10if")
_BLOCK_ATTEND = struct.Struct("@PqPPPPPPPPPPN10if")
_PAGE_POOL = struct.Struct("@PPN2i")
KV_FORMATS = {"native": 0, "e4m3": 1, "e2m1": 2}
MAX_STEP_BATCH = 1024


_lib = None


def lib(build_if_missing: bool = False):
    """The loaded libdkv (built in-tree by ``zero_copy_offloaded_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise ImportError(f"{path} is missing: run zero_copy_offloaded_gb300/build.py "
                              "(the CUDA library is required; there is no fallback)")
        from . import build as _b
        _b.build()
    L = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "dkv_cache_alloc": [ctypes.POINTER(P), I, I, I, I, I],
        "dkv_cache_alloc_paged": [ctypes.POINTER(P), I, I, I, I, I, I, I],
        "dkv_cache_set_page_table": [P, P],
        "dkv_cache_alloc_layered": [ctypes.POINTER(P), I, I, I, I, I, I],
        "dkv_cache_alloc_ex": [ctypes.POINTER(P), ctypes.POINTER(_CacheDesc)],
        "dkv_decode_layer": [P, I, P, P, P, P, I, I, P, P],
        "dkv_prefill_layer": [P, I, P, I, P, P, P, I, I, P, P],
        "dkv_step_graph_capture": [P, I, I, P, P, P, P, P],
        "dkv_step_graph_launch": [P, P],
        "dkv_free": [P],
        "dkv_cache_host_ptrs": [P, ctypes.POINTER(P), ctypes.POINTER(P)],
        "dkv_cache_device_ptrs": [P, ctypes.POINTER(P), ctypes.POINTER(P)],
        "dkv_cache_set_lengths": [P, P],
        "dkv_cache_get_lengths": [P, P],
        "dkv_cache_info": [P, ctypes.POINTER(_CacheInfo)],
        "dkv_cache_reserve": [P, I, I],
        "dkv_cache_set_tuning": [P, I, I, I],
        "dkv_decode": [P, P, P, P, P, I, I, P, P],
        "dkv_prefill": [P, P, I, P, P, P, I, I, P, P],
        "dkv_sync_status": [P, P],
        "dkv_probe_read": [P, Z, P, P],
        "dkv_probe_write": [P, Z, P],
        "dkv_probe_launch": [I, I, I, P],
        "dkv_attend_naive": [P, P, I, P, P],
        "dkv_decode_staged": [P, P, P, P, P, I, I, P, P, P, P],
        "dkv_prefill_staged": [P, P, I, P, P, P, I, I, P, P, P, P],
        "dkv_prefill_naive": [P, P, I, P, P, P, I, I, P, P],
        "dkv_decode_unfused": [P, P, P, P, P, I, I, P, P],
        "dkv_cache_kernel_timing": [P, I],
        "dkv_cache_last_kernel_ms": [P, ctypes.POINTER(ctypes.c_float)],
        "dkv_decode_noalloc": [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P],
        "dkv_decode_noalloc_status": [P],
        "dkv_decode_noalloc_debug_withhold": [I],
        "dkv_step_plan": [P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, P, P],
        "dkv_qkv_append": [P, P],
        "dkv_paged_attend": [P, P],
        "dkv_paged_attend_debug_withhold": [I],
        "dkv_block_append": [P, P],
        "dkv_block_attend": [P, P],
        "dkv_pages_fork": [P] * 5 + [I] * 4 + [P] * 6 + [Z, P],
        "dkv_pages_compact": [P, P, I, I, I, I, P, P, P, P, I, P, P, Z, P],
        "dkv_pages_copy": [P, I, P, I, P],
        "dkv_project": [P, P, P, I, I, I, I, P],
        "dkv_cache_debug_withhold": [P, I],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    L.dkv_status_str.argtypes = [ctypes.c_int]
    L.dkv_status_str.restype = ctypes.c_char_p
    L.dkv_last_error.argtypes = []
    L.dkv_last_error.restype = ctypes.c_char_p
    L.dkv_last_launch_count.argtypes = []
    L.dkv_last_launch_count.restype = ctypes.c_int
    L.dkv_pci_numa_node.argtypes = [ctypes.c_char_p, ctypes.c_char_p]
    L.dkv_pci_numa_node.restype = ctypes.c_int
    L.dkv_stream_capturing.argtypes = [P]
    L.dkv_stream_capturing.restype = ctypes.c_int
    L.dkv_paged_attend_workspace.argtypes = [I] * 5
    L.dkv_paged_attend_workspace.restype = ctypes.c_size_t
    L.dkv_pages_workspace.argtypes = [I] * 3
    L.dkv_pages_workspace.restype = ctypes.c_size_t
    L.dkv_numa_probe.argtypes = [ctypes.c_int]
    L.dkv_numa_probe.restype = ctypes.c_int
    _lib = L
    return L


def _check(st: int, where: str):
    if st != 0:
        raise DkvError(st, where, lib().dkv_last_error().decode())


def _ptr(t) -> int | None:
    """Device pointer of a CUDA tensor (or an int / None passed through)."""
    if t is None or isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return t.data_ptr()
    raise TypeError(f"cannot take a device pointer of {type(t)}")


def _stream(s) -> int | None:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def dkv_status_str(st: int) -> str:
    return lib().dkv_status_str(st).decode()


def dkv_last_error() -> str:
    return lib().dkv_last_error().decode()


def dkv_last_launch_count() -> int:
    return lib().dkv_last_launch_count()


def dkv_cache_alloc(batch, n_kv_heads, head_dim, max_tokens, dtype="bf16") -> int:
    h = ctypes.c_void_p()
    _check(lib().dkv_cache_alloc(ctypes.byref(h), batch, n_kv_heads, head_dim, max_tokens,
                                 _DTYPE[dtype]), "dkv_cache_alloc")
    return h.value


def dkv_cache_alloc_paged(batch, n_kv_heads, head_dim, page_tokens, num_pages,
                          max_pages_per_seq, dtype="bf16") -> int:
    h = ctypes.c_void_p()
    _check(lib().dkv_cache_alloc_paged(ctypes.byref(h), batch, n_kv_heads, head_dim, page_tokens,
                                       num_pages, max_pages_per_seq, _DTYPE[dtype]),
           "dkv_cache_alloc_paged")
    return h.value


def dkv_cache_set_page_table(h, table):
    """table: int32 [batch, max_pages_per_seq] of pool page indices (-1: none)."""
    t = np.ascontiguousarray(table, dtype=np.int32)
    _check(lib().dkv_cache_set_page_table(h, t.ctypes.data), "dkv_cache_set_page_table")


def dkv_cache_alloc_ex(batch, n_kv_heads, head_dim, max_tokens=0, dtype="bf16",
                       kv_format="native", layers=1, page_tokens=0, num_pages=0,
                       max_pages_per_seq=0) -> int:
    d = _CacheDesc(batch, n_kv_heads, head_dim, max_tokens, _DTYPE[dtype], KV_FORMATS[kv_format],
                   layers, page_tokens, num_pages, max_pages_per_seq)
    h = ctypes.c_void_p()
    _check(lib().dkv_cache_alloc_ex(ctypes.byref(h), ctypes.byref(d)), "dkv_cache_alloc_ex")
    return h.value


def dkv_cache_alloc_layered(layers, batch, n_kv_heads, head_dim, max_tokens, dtype="bf16") -> int:
    h = ctypes.c_void_p()
    _check(lib().dkv_cache_alloc_layered(ctypes.byref(h), layers, batch, n_kv_heads, head_dim,
                                         max_tokens, _DTYPE[dtype]), "dkv_cache_alloc_layered")
    return h.value


def dkv_decode_layer(h, layer, x, wq, wk, wv, hidden, n_q_heads, out, stream=None):
    _check(lib().dkv_decode_layer(h, layer, _ptr(x), _ptr(wq), _ptr(wk), _ptr(wv), hidden,
                                  n_q_heads, _ptr(out), _stream(stream)), "dkv_decode_layer")


def dkv_prefill_layer(h, layer, x, T, wq, wk, wv, hidden, n_q_heads, out, stream=None):
    _check(lib().dkv_prefill_layer(h, layer, _ptr(x), T, _ptr(wq), _ptr(wk), _ptr(wv), hidden,
                                   n_q_heads, _ptr(out), _stream(stream)), "dkv_prefill_layer")


def _ptr_array(ts):
    arr = (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])
    return arr


def dkv_step_graph_capture(h, hidden, n_q_heads, xs, wqs, wks, wvs, outs):
    """Per-layer lists of device tensors; the arrays are copied into the graph."""
    arrs = [_ptr_array(v) for v in (xs, wqs, wks, wvs, outs)]
    _check(lib().dkv_step_graph_capture(h, hidden, n_q_heads,
                                        *[ctypes.cast(a, ctypes.c_void_p) for a in arrs]),
           "dkv_step_graph_capture")


def dkv_step_graph_launch(h, stream=None):
    _check(lib().dkv_step_graph_launch(h, _stream(stream)), "dkv_step_graph_launch")


def dkv_free(h):
    _check(lib().dkv_free(h), "dkv_free")


def dkv_cache_host_ptrs(h):
    k, v = ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib().dkv_cache_host_ptrs(h, ctypes.byref(k), ctypes.byref(v)), "dkv_cache_host_ptrs")
    return k.value, v.value


def dkv_cache_device_ptrs(h):
    k, v = ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib().dkv_cache_device_ptrs(h, ctypes.byref(k), ctypes.byref(v)),
           "dkv_cache_device_ptrs")
    return k.value, v.value


def dkv_cache_set_lengths(h, lens):
    a = np.ascontiguousarray(lens, dtype=np.int32)
    _check(lib().dkv_cache_set_lengths(h, a.ctypes.data), "dkv_cache_set_lengths")


def dkv_cache_get_lengths(h, batch):
    a = np.zeros(batch, np.int32)
    _check(lib().dkv_cache_get_lengths(h, a.ctypes.data), "dkv_cache_get_lengths")
    return a


def dkv_cache_info(h) -> dict:
    i = _CacheInfo()
    _check(lib().dkv_cache_info(h, ctypes.byref(i)), "dkv_cache_info")
    return {f: getattr(i, f) for f, _ in _CacheInfo._fields_}


def dkv_pci_numa_node(pci_bus_id: str, sysfs_root: str | None = None) -> int:
    """Host NUMA node of a PCI device (-1 if unknown); see include/dkv.h."""
    return lib().dkv_pci_numa_node(pci_bus_id.encode(),
                                   sysfs_root.encode() if sysfs_root else None)


def dkv_numa_probe(node: int) -> int:
    return lib().dkv_numa_probe(int(node))


def dkv_cache_reserve(h, n_q_heads, max_new_tokens):
    _check(lib().dkv_cache_reserve(h, n_q_heads, max_new_tokens), "dkv_cache_reserve")


def dkv_cache_set_tuning(h, splits=0, tile_n=0, stages=0):
    _check(lib().dkv_cache_set_tuning(h, splits, tile_n, stages), "dkv_cache_set_tuning")


def dkv_cache_debug_withhold(h, enable=True):
    _check(lib().dkv_cache_debug_withhold(h, int(bool(enable))), "dkv_cache_debug_withhold")


def dkv_cache_kernel_timing(h, enable=True):
    _check(lib().dkv_cache_kernel_timing(h, int(bool(enable))), "dkv_cache_kernel_timing")


def dkv_cache_last_kernel_ms(h) -> float:
    ms = ctypes.c_float()
    _check(lib().dkv_cache_last_kernel_ms(h, ctypes.byref(ms)), "dkv_cache_last_kernel_ms")
    return float(ms.value)


def dkv_decode(h, x, wq, wk, wv, hidden, n_q_heads, out, stream=None):
    _check(lib().dkv_decode(h, _ptr(x), _ptr(wq), _ptr(wk), _ptr(wv), hidden, n_q_heads,
                            _ptr(out), _stream(stream)), "dkv_decode")


def dkv_prefill(h, x, T, wq, wk, wv, hidden, n_q_heads, out, stream=None):
    _check(lib().dkv_prefill(h, _ptr(x), T, _ptr(wq), _ptr(wk), _ptr(wv), hidden, n_q_heads,
                             _ptr(out), _stream(stream)), "dkv_prefill")


def dkv_sync_status(h, stream=None):
    _check(lib().dkv_sync_status(h, _stream(stream)), "dkv_sync_status")


def dkv_project(x, w, y, M, K, N, dtype="bf16", stream=None):
    _check(lib().dkv_project(_ptr(x), _ptr(w), _ptr(y), M, K, N, _DTYPE[dtype], _stream(stream)),
           "dkv_project")


def dkv_probe_read(src, nbytes, sink, stream=None):
    _check(lib().dkv_probe_read(_ptr(src), nbytes, _ptr(sink), _stream(stream)), "dkv_probe_read")


def dkv_probe_write(dst, nbytes, stream=None):
    _check(lib().dkv_probe_write(_ptr(dst), nbytes, _stream(stream)), "dkv_probe_write")


def dkv_probe_launch(grid, threads, smem_bytes, stream=None):
    _check(lib().dkv_probe_launch(grid, threads, smem_bytes, _stream(stream)), "dkv_probe_launch")


def dkv_attend_naive(h, q, n_q_heads, out, stream=None):
    _check(lib().dkv_attend_naive(h, _ptr(q), n_q_heads, _ptr(out), _stream(stream)),
           "dkv_attend_naive")


def dkv_decode_unfused(h, x, wq, wk, wv, hidden, n_q_heads, out, stream=None):
    _check(lib().dkv_decode_unfused(h, _ptr(x), _ptr(wq), _ptr(wk), _ptr(wv), hidden, n_q_heads,
                                    _ptr(out), _stream(stream)), "dkv_decode_unfused")


def dkv_decode_staged(h, x, wq, wk, wv, hidden, n_q_heads, out, k_stage, v_stage, stream=None):
    _check(lib().dkv_decode_staged(h, _ptr(x), _ptr(wq), _ptr(wk), _ptr(wv), hidden, n_q_heads,
                                   _ptr(out), _ptr(k_stage), _ptr(v_stage), _stream(stream)),
           "dkv_decode_staged")


def dkv_prefill_staged(h, x, T, wq, wk, wv, hidden, n_q_heads, out, k_stage, v_stage,
                       stream=None):
    _check(lib().dkv_prefill_staged(h, _ptr(x), T, _ptr(wq), _ptr(wk), _ptr(wv), hidden,
                                    n_q_heads, _ptr(out), _ptr(k_stage), _ptr(v_stage),
                                    _stream(stream)),
           "dkv_prefill_staged")


def dkv_prefill_naive(h, x, T, wq, wk, wv, hidden, n_q_heads, out, stream=None):
    _check(lib().dkv_prefill_naive(h, _ptr(x), T, _ptr(wq), _ptr(wk), _ptr(wv), hidden,
                                   n_q_heads, _ptr(out), _stream(stream)),
           "dkv_prefill_naive")


def dkv_decode_noalloc(x, wq, wk, wv, k_cache, v_cache, lengths, batch, hidden, n_q_heads,
                       n_kv_heads, head_dim, max_tokens, dtype, out, stream=None):
    """dkv_decode on caller-owned buffers with no allocation (see include/dkv.h)."""
    lens = np.ascontiguousarray(lengths, dtype=np.int32).reshape(-1)
    if lens.size < batch:
        raise ValueError(f"lengths holds {lens.size} entries for a batch of {batch}")
    _check(lib().dkv_decode_noalloc(_ptr(x), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(k_cache),
                                    _ptr(v_cache), lens.ctypes.data, batch, hidden, n_q_heads,
                                    n_kv_heads, head_dim, max_tokens, _DTYPE[dtype], _ptr(out),
                                    _stream(stream)), "dkv_decode_noalloc")


def dkv_decode_noalloc_status(stream=None):
    """Status of the last dkv_decode_noalloc on the current device (raises on an error)."""
    _check(lib().dkv_decode_noalloc_status(_stream(stream)), "dkv_decode_noalloc_status")


def dkv_decode_noalloc_debug_withhold(enable=True):
    _check(lib().dkv_decode_noalloc_debug_withhold(int(bool(enable))),
           "dkv_decode_noalloc_debug_withhold")


# ---- the device-side step over a 4-bit paged cache -----------------------------------

def _bad(t, what, dtype, index, shape):
    if t.dtype != dtype:
        raise ValueError(f"{what} is {t.dtype}, not {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{what} is on {t.device}, not with the others")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {shape}")
    raise ValueError(f"{what} must be contiguous")


def _arg(t, what, dtype, index, shape=None):
    """Address of a contiguous tensor of this dtype, device index and shape; 0 for None."""
    if t is None:
        return 0
    if (t.dtype is not dtype or t.get_device() != index or not t.is_contiguous()
            or (shape is not None and t.shape != shape)):
        _bad(t, what, dtype, index, shape)
    return t.data_ptr()


def _rows(t, what, dtype, index, rows, D):
    """Address, heads and token stride of [rows, heads, D] whose heads are contiguous in each row."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != rows or shape[2] != D:
        raise ValueError(f"{what} has shape {tuple(shape)}: [{rows}, heads, {D}] is wanted")
    if t.dtype != dtype or t.get_device() != index:
        _bad(t, what, dtype, index, None)
    h, st = shape[1], t.stride()
    if st[2] != 1 or (h > 1 and st[1] != D):
        raise ValueError(f"the heads of a row of {what} must be contiguous")
    return t.data_ptr(), h, (st[0] if rows > 1 else h * D)


def _pool(t, what, u8, index, D):
    """Address and (num_pages, n_kv_heads, page_tokens) of an E2M1 pool: CUDA, or pinned host memory."""
    shape = t.shape
    if t.dtype != u8 or len(shape) != 3 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous uint8 [num_pages, n_kv_heads, page bytes]")
    if t.get_device() != index and not (t.get_device() < 0 and t.is_pinned()):
        raise ValueError(f"{what} is neither with the other tensors nor in pinned host memory")
    pages, heads, nbytes = shape
    per = D * 9 // 16
    if nbytes % per:
        raise ValueError(f"{what}: a page of {nbytes} bytes does not hold rows of {per}")
    return t.data_ptr(), (pages, heads, nbytes // per)


@functools.lru_cache(maxsize=None)
def _torch_calls():
    """torch's current device, raw current stream of a device, and its allocator's allocate (size, raw stream)
    and free: the calls inside its public ones, which take 1 to 3 us more of the 10 that the smallest
    operators take, or the public ones where a release does not have them."""
    import torch
    c, cuda = torch._C, torch.cuda
    return (getattr(c, "_cuda_getDevice", cuda.current_device),
            getattr(c, "_cuda_getCurrentRawStream", lambda index: cuda.current_stream(index).cuda_stream),
            getattr(c, "_cuda_cudaCachingAllocator_raw_alloc",
                    lambda size, stream: cuda.caching_allocator_alloc(size, stream=stream)),
            getattr(c, "_cuda_cudaCachingAllocator_raw_delete", cuda.caching_allocator_delete))


def _launch(index, stream):
    """The stream to launch on; the tensors must be on the current device, as the library launches there."""
    device, current, _, _ = _torch_calls()
    if index < 0 or index != device():  # a CUDA tensor is there: torch is set up
        raise ValueError("the tensors are not on the current CUDA device")
    if stream is None:
        return current(index)
    return _stream(stream)


def rope_table(max_positions, rotary_dim, base=10000.0, device="cuda"):
    """fp32 [max_positions, rotary_dim]: the cosines, then the sines, of position * base^(-2i/rotary_dim),
    from angles in 64 bits."""
    import torch
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device)
    a = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * base ** (-i / rotary_dim)
    return torch.cat((a.cos(), a.sin()), -1).to(torch.float32)


def dkv_step_plan(lengths, new_tokens, page_table, free_pages, free_count, page_tokens, row_start,
                  row_pos, row_slot, kv_len, free_left, report, stream=None):
    """Pages, row starts, positions and slots of a step from its lengths, on the GPU (see
    include/dkv.h).  All tensors are int32 and CUDA; page_table [batch, max_pages], row_pos and
    row_slot [max_rows], report [4]."""
    import torch
    i32 = torch.int32
    if page_table.dim() != 2 or row_pos.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("page_table is [batch, max_pages], row_pos [max_rows], free_pages [num_pages]")
    B, max_pages = page_table.shape
    n, pages, dev = row_pos.shape[0], free_pages.shape[0], page_table.get_device()
    each, one = (B,), (1,)
    st = lib().dkv_step_plan(
        _arg(lengths, "lengths", i32, dev, each), _arg(new_tokens, "new_tokens", i32, dev, each),
        _arg(page_table, "page_table", i32, dev), _arg(free_pages, "free_pages", i32, dev),
        _arg(free_count, "free_count", i32, dev, one), B, max_pages, page_tokens, pages, n,
        _arg(row_start, "row_start", i32, dev, (B + 1,)), _arg(row_pos, "row_pos", i32, dev),
        _arg(row_slot, "row_slot", i32, dev, (n,)), _arg(kv_len, "kv_len", i32, dev, each),
        _arg(free_left, "free_left", i32, dev, one), _arg(report, "report", i32, dev, (4,)),
        _launch(dev, stream))
    if st:
        _check(st, "dkv_step_plan")


def _dtype_of(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return FP16
    raise ValueError(f"{t.dtype} is neither bfloat16 nor float16")


def _append_args(q, k, v, positions, slots, q_out, k_out, v_out, q_gamma, k_gamma, cos_sin):
    """What the appends check alike: the device index, the fields of dkv_append_t but the pools and what comes behind
    max_positions, in their order.  (One flat tuple: nested ones cost the smallest calls a microsecond of their ten.)"""
    import torch
    some = q if q is not None else k
    if some is None:
        raise ValueError("neither queries nor keys")
    if some.dim() != 3:
        raise ValueError("q, k and v are [rows, heads, head_dim]")
    dev, dt, code = some.get_device(), some.dtype, _dtype_of(some)
    n, _, D = some.shape
    i32, f32 = torch.int32, torch.float32
    pq = hq = sq = pqo = pqg = pk = pv = hkv = sk = sv = pko = pvo = pkg = 0
    if q is not None:
        pq, hq, sq = _rows(q, "q", dt, dev, n, D)
        pqo = _arg(q_out, "q_out", dt, dev, (n, hq, D))
        pqg = _arg(q_gamma, "q_gamma", dt, dev, (D,))
    if k is not None:
        if v is None or v.shape != k.shape:
            raise ValueError("k and v are both [rows, n_kv_heads, head_dim]")
        pk, hkv, sk = _rows(k, "k", dt, dev, n, D)
        pv, _, sv = _rows(v, "v", dt, dev, n, D)
        pko = _arg(k_out, "k_out", dt, dev, (n, hkv, D))
        pvo = _arg(v_out, "v_out", dt, dev, (n, hkv, D))
        pkg = _arg(k_gamma, "k_gamma", dt, dev, (D,))
    elif v is not None:
        raise ValueError("keys and values come together")
    pcs = pp = max_positions = rotary_dim = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin is [max_positions, rotary_dim]")
        pcs = _arg(cos_sin, "cos_sin", f32, dev)
        max_positions, rotary_dim = cos_sin.shape
        pp = _arg(positions, "positions", i32, dev, (n,))
    return (dev, pq, pk, pv, sq, sk, sv, pqg, pkg, pcs, pp, _arg(slots, "slots", i32, dev, (n,)), pqo, pko, pvo,
            n, hq, hkv, D, code, rotary_dim, max_positions)


def dkv_qkv_append(q, k, v, positions=None, slots=None, k_pool=None, v_pool=None, q_out=None,
                   k_out=None, v_out=None, q_gamma=None, k_gamma=None, eps=1e-6, cos_sin=None,
                   interleaved=False, k_scale=1.0, v_scale=1.0, stream=None):
    """Head norms and rotation of q and k, append of k and v to an E2M1 pool (see include/dkv.h).
    q [rows, n_q_heads, D] and k, v [rows, n_kv_heads, D] may be slices of one projection's output."""
    import torch
    (dev, pq, pk, pv, sq, sk, sv, pqg, pkg, pcs, pp, ps, pqo, pko, pvo, n, hq, hkv, D, code, rotary_dim,
     max_positions) = _append_args(q, k, v, positions, slots, q_out, k_out, v_out, q_gamma, k_gamma, cos_sin)
    pkp = pvp = pages = page_tokens = 0
    if k_pool is not None:
        if v_pool is None or k is None:
            raise ValueError("both pools and the keys come together")
        pkp, shape = _pool(k_pool, "k_pool", torch.uint8, dev, D)
        pvp, other = _pool(v_pool, "v_pool", torch.uint8, dev, D)
        if shape != other or shape[1] != hkv:
            raise ValueError(f"pools of {shape} and {other} (pages, heads, page_tokens) for {hkv} heads")
        pages, page_tokens = shape[0], shape[2]
    st = lib().dkv_qkv_append(
        _APPEND.pack(pq, pk, pv, sq, sk, sv, pqg, pkg, pcs, pp, ps, pkp, pvp, pqo, pko, pvo, n, hq, hkv, D, code,
                     rotary_dim, max_positions, bool(interleaved), page_tokens, pages, eps, k_scale, v_scale),
        _launch(dev, stream))
    if st:
        _check(st, "dkv_qkv_append")


def _near(t, what, index):
    """Address of a contiguous tensor on this device, or in pinned host memory."""
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.get_device() != index and not (t.get_device() < 0 and t.is_pinned()):
        raise ValueError(f"{what} is neither with the other tensors nor in pinned host memory")
    return t.data_ptr()


def _block_pools(k_pool, v_pool, k_scales, v_scales, index, D):
    """Addresses of the pools and scales of an 8-bit cache, num_pages, n_kv_heads and page_tokens."""
    import torch
    shape = k_pool.shape
    if len(shape) != 4 or shape[3] != D or v_pool.shape != shape:
        raise ValueError(f"pools of {tuple(shape)} and {tuple(v_pool.shape)}: both are [num_pages, n_kv_heads, page_tokens, {D}]")
    pages, heads, page_tokens, _ = shape
    for t, what in ((k_pool, "k_pool"), (v_pool, "v_pool")):
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError(f"{what} is {t.dtype}, neither float8_e4m3fn nor its bytes (uint8)")
    for t, what in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        if t.dtype != torch.float32 or page_tokens % 16 or t.shape != (pages, heads, page_tokens // 16):
            raise ValueError(f"{what} is {t.dtype} {tuple(t.shape)}: float32 [{pages}, {heads}, {page_tokens} / 16] is wanted")
    return (_near(k_pool, "k_pool", index), _near(v_pool, "v_pool", index), _near(k_scales, "k_scales", index),
            _near(v_scales, "v_scales", index), pages, heads, page_tokens)


def dkv_block_append(q, k, v, positions, slots, k_pool, v_pool, k_scales, v_scales, q_out=None, k_out=None, v_out=None,
                     q_gamma=None, k_gamma=None, eps=1e-6, cos_sin=None, interleaved=False, stream=None):
    """dkv_qkv_append into an 8-bit pool with block scales (see include/dkv.h): k_pool, v_pool float8_e4m3fn
    [num_pages, n_kv_heads, page_tokens, D], k_scales, v_scales fp32 [num_pages, n_kv_heads, page_tokens // 16].  q may
    be None."""
    (dev, pq, pk, pv, sq, sk, sv, pqg, pkg, pcs, pp, ps, pqo, pko, pvo, n, hq, hkv, D, code, rotary_dim,
     max_positions) = _append_args(q, k, v, positions, slots, q_out, k_out, v_out, q_gamma, k_gamma, cos_sin)
    pkp, pvp, pks, pvs, pages, heads, page_tokens = _block_pools(k_pool, v_pool, k_scales, v_scales, dev, D)
    if k is None or heads != hkv:
        raise ValueError(f"pools of {(pages, heads, page_tokens)} (pages, heads, page_tokens) for {hkv} heads")
    st = lib().dkv_block_append(
        _BLOCK_APPEND.pack(pq, pk, pv, sq, sk, sv, pqg, pkg, pcs, pp, ps, pkp, pvp, pks, pvs, pqo, pko, pvo, n, hq, hkv,
                           D, code, rotary_dim, max_positions, bool(interleaved), page_tokens, pages, eps),
        _launch(dev, stream))
    if st:
        _check(st, "dkv_block_append")


@functools.lru_cache(maxsize=256)
def dkv_paged_attend_workspace(batch, n_q_heads, n_kv_heads, head_dim, max_rows=1) -> int:
    """Bytes of device memory that dkv_paged_attend needs (0 for arguments that it refuses)."""
    return lib().dkv_paged_attend_workspace(batch, n_q_heads, n_kv_heads, head_dim, max_rows)


def _kept_for_graph(address):
    """Whether torch's allocator keeps this address for a graph: in a pool of its own, as it does for the graphs that
    torch captures, or (other allocators) as a node of the graph."""
    import torch
    if torch.cuda.get_allocator_backend() != "native":
        return True
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= address < s["address"] + s["total_size"]:
            return tuple(s["segment_pool_id"]) != (0, 0)
    return False


def _take(size, s):
    """Address of a workspace from torch's allocator, which the caller releases once the call is enqueued.  The
    allocator's own call: a tensor around the bytes costs 3 us of the smallest calls' 13.  The bytes are the launching
    stream's, so that they are not handed out again before it ran."""
    _, _, allocate, release = _torch_calls()
    taken = allocate(max(1, size), s)
    if lib().dkv_stream_capturing(s) == 1 and not _kept_for_graph(taken):
        # the allocator would hand the bytes out again while the graph lives
        release(taken)
        raise ValueError("a stream capture that torch does not know needs a workspace of its own")
    return taken


def _attend_args(q, page_table, kv_len, out, row_start, lse, stream):
    """What the attentions check alike: device index, stream, address of q and its stride, addresses of page_table, kv_len,
    row_start, out and lse, batch, rows, query heads, head_dim, dtype code and max_pages."""
    import torch
    shape, i32 = q.shape, torch.int32
    if len(shape) != 3 or page_table.dim() != 2:
        raise ValueError("q is [rows, n_q_heads, head_dim], page_table [batch, max_pages]")
    dev, dt = q.get_device(), q.dtype
    code = _dtype_of(q)
    s = _launch(dev, stream)
    n, _, D = shape
    pq, hq, sq = _rows(q, "q", dt, dev, n, D)
    B, max_pages = page_table.shape
    return (dev, s, pq, sq, _arg(page_table, "page_table", i32, dev), _arg(kv_len, "kv_len", i32, dev, (B,)),
            _arg(row_start, "row_start", i32, dev, (B + 1,)), _arg(out, "out", dt, dev, (n, hq, D)),
            _arg(lse, "lse", torch.float32, dev, (n, hq)), B, n, hq, D, code, max_pages)


def dkv_paged_attend(q, k_pool, v_pool, page_table, kv_len, out, row_start=None, max_rows=1,
                     scale=None, v_scale=1.0, lse=None, workspace=None, stream=None):
    """Attention of q [rows, n_q_heads, D] over an E2M1 pool (see include/dkv.h); scale None is
    1/sqrt(D).  Without a workspace (uint8, dkv_paged_attend_workspace bytes) one is taken from
    torch's caching allocator, on the launching stream; under a stream capture that is not torch's
    own (torch.cuda.graph) the call needs one, which the graph's owner keeps."""
    import torch
    dev, s, pq, sq, pt, pkl, prs, po, pl, B, n, hq, D, code, max_pages = _attend_args(
        q, page_table, kv_len, out, row_start, lse, stream)
    pkp, shape = _pool(k_pool, "k_pool", torch.uint8, dev, D)
    pvp, other = _pool(v_pool, "v_pool", torch.uint8, dev, D)
    if shape != other:
        raise ValueError(f"pools of {shape} and {other} (pages, heads, page_tokens)")
    pages, hkv, page_tokens = shape
    if workspace is None:
        size = dkv_paged_attend_workspace(B, hq, hkv, D, max_rows)
        pw = _take(size, s)
    else:
        pw, size = _arg(workspace, "workspace", torch.uint8, dev), workspace.numel()
    try:
        st = lib().dkv_paged_attend(
            _ATTEND.pack(pq, sq, pkp, pvp, pt, pkl, prs, po, pl, pw, size, B, n, max_rows, hq, hkv, D, code,
                         page_tokens, pages, max_pages, D ** -0.5 if scale is None else scale, v_scale), s)
    finally:
        if workspace is None:
            _torch_calls()[3](pw)
    if st:
        _check(st, "dkv_paged_attend")


def dkv_block_attend(q, k_pool, v_pool, k_scales, v_scales, page_table, kv_len, out, row_start=None, max_rows=1,
                     scale=None, lse=None, workspace=None, stream=None):
    """dkv_paged_attend over an 8-bit pool with block scales (see include/dkv.h), as dkv_block_append fills it."""
    import torch
    dev, s, pq, sq, pt, pkl, prs, po, pl, B, n, hq, D, code, max_pages = _attend_args(
        q, page_table, kv_len, out, row_start, lse, stream)
    pkp, pvp, pks, pvs, pages, hkv, page_tokens = _block_pools(k_pool, v_pool, k_scales, v_scales, dev, D)
    if workspace is None:
        size = dkv_paged_attend_workspace(B, hq, hkv, D, max_rows)
        pw = _take(size, s)
    else:
        pw, size = _arg(workspace, "workspace", torch.uint8, dev), workspace.numel()
    try:
        st = lib().dkv_block_attend(
            _BLOCK_ATTEND.pack(pq, sq, pkp, pvp, pks, pvs, pt, pkl, prs, po, pl, pw, size, B, n, max_rows, hq, hkv, D,
                               code, page_tokens, pages, max_pages, D ** -0.5 if scale is None else scale), s)
    finally:
        if workspace is None:
            _torch_calls()[3](pw)
    if st:
        _check(st, "dkv_block_attend")


def dkv_paged_attend_debug_withhold(enable=True):
    _check(lib().dkv_paged_attend_debug_withhold(int(bool(enable))), "dkv_paged_attend_debug_withhold")


# ---- the life of a cache's pages -----------------------------------------------------

@functools.lru_cache(maxsize=256)
def dkv_pages_workspace(batch, max_pages, num_pages) -> int:
    """Bytes of device memory that dkv_pages_fork and dkv_pages_compact need (0 for sizes that they refuse)."""
    return lib().dkv_pages_workspace(batch, max_pages, num_pages)


def dkv_pages_fork(page_table, kv_len, sources, free_pages, free_count, page_tokens, table_out, len_out, free_left,
                   copies, report, workspace=None, stream=None):
    """Sequence b becomes a copy of sequence sources[b], or ends (see include/dkv.h).  All tensors are int32 and
    CUDA; page_table and table_out [batch, max_pages], free_pages [num_pages], copies [batch, 2], report [4].
    Without a workspace (uint8, dkv_pages_workspace bytes) one is taken as dkv_paged_attend does."""
    import torch
    i32 = torch.int32
    if page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("page_table is [batch, max_pages], free_pages [num_pages]")
    B, max_pages = page_table.shape
    pages, dev, each, one = free_pages.shape[0], page_table.get_device(), (B,), (1,)
    s = _launch(dev, stream)
    args = (_arg(page_table, "page_table", i32, dev), _arg(kv_len, "kv_len", i32, dev, each),
            _arg(sources, "sources", i32, dev, each), _arg(free_pages, "free_pages", i32, dev),
            _arg(free_count, "free_count", i32, dev, one), B, max_pages, page_tokens, pages,
            _arg(table_out, "table_out", i32, dev, (B, max_pages)), _arg(len_out, "len_out", i32, dev, each),
            _arg(free_left, "free_left", i32, dev, one), _arg(copies, "copies", i32, dev, (B, 2)),
            _arg(report, "report", i32, dev, (4,)))
    if workspace is None:
        size = dkv_pages_workspace(B, max_pages, pages)
        pw = _take(size, s)
    else:
        pw, size = _arg(workspace, "workspace", torch.uint8, dev), workspace.numel()
    try:
        st = lib().dkv_pages_fork(*args, pw, size, s)
    finally:
        if workspace is None:
            _torch_calls()[3](pw)
    if st:
        _check(st, "dkv_pages_fork")


def dkv_pages_compact(page_table, kv_len, page_tokens, table_out, free_pages, free_left, moves, report,
                      workspace=None, stream=None):
    """The pages held move to the front of the pool of free_pages.shape[0] pages (see include/dkv.h).  All tensors are
    int32 and CUDA; moves [at least num_pages // 2, 2], report [4]."""
    import torch
    i32 = torch.int32
    if page_table.dim() != 2 or free_pages.dim() != 1 or moves.dim() != 2 or moves.shape[1] != 2:
        raise ValueError("page_table is [batch, max_pages], free_pages [num_pages], moves [max_moves, 2]")
    B, max_pages = page_table.shape
    pages, dev = free_pages.shape[0], page_table.get_device()
    s = _launch(dev, stream)
    args = (_arg(page_table, "page_table", i32, dev), _arg(kv_len, "kv_len", i32, dev, (B,)), B, max_pages,
            page_tokens, pages, _arg(table_out, "table_out", i32, dev, (B, max_pages)),
            _arg(free_pages, "free_pages", i32, dev), _arg(free_left, "free_left", i32, dev, (1,)),
            _arg(moves, "moves", i32, dev), moves.shape[0], _arg(report, "report", i32, dev, (4,)))
    if workspace is None:
        size = dkv_pages_workspace(B, max_pages, pages)
        pw = _take(size, s)
    else:
        pw, size = _arg(workspace, "workspace", torch.uint8, dev), workspace.numel()
    try:
        st = lib().dkv_pages_compact(*args, pw, size, s)
    finally:
        if workspace is None:
            _torch_calls()[3](pw)
    if st:
        _check(st, "dkv_pages_compact")


def dkv_pages_copy(pairs, pools, into=None, stream=None):
    """Page pairs[i, 1] of each tensor of `into` takes the bytes of page pairs[i, 0] of the tensor of `pools` beside it
    (see include/dkv.h).  pairs: int32 CUDA [n, 2], {-1, -1} for nothing.  pools, into: lists of contiguous
    tensors [pages, ...], CUDA or in pinned host memory; into None: the same pools."""
    import torch
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs is [n, 2]")
    dev = pairs.get_device()
    into = pools if into is None else into
    if len(into) != len(pools):
        raise ValueError(f"{len(pools)} pools into {len(into)}")
    packed = bytearray()
    for i, (a, b) in enumerate(zip(pools, into)):
        shape = a.shape
        if len(shape) < 2 or a is not b and (a.dtype != b.dtype or shape[1:] != b.shape[1:]):
            raise ValueError(f"pool {i}: {a.dtype} {tuple(a.shape)} does not go into {b.dtype} {tuple(b.shape)}")
        to = at = _near(a, f"pool {i}", dev)
        count = n = shape[0]
        if a is not b:
            to, count = _near(b, f"pool {i}", dev), b.shape[0]
        packed += _PAGE_POOL.pack(at, to, a.nbytes // n if n else 0, n, count)
    n = pairs.shape[0]
    st = lib().dkv_pages_copy(_arg(pairs, "pairs", torch.int32, dev), n,
                              ctypes.addressof(ctypes.c_char.from_buffer(packed)) if packed else None, len(pools),
                              _launch(dev, stream))
    if st:
        _check(st, "dkv_pages_copy")


class KVCache:
    """Owner of one dkv_cache handle, with numpy views of the pinned caches."""

    def __init__(self, batch, n_kv_heads, head_dim, max_tokens, dtype="bf16", kv_format="native"):
        """kv_format "e4m3": 8-bit E4M3 elements (views of uint8 bits; decode only)."""
        self.B, self.Hkv, self.D, self.S_max = batch, n_kv_heads, head_dim, max_tokens
        self.dtype, self.kv_format = dtype, kv_format
        self.h = dkv_cache_alloc_ex(batch, n_kv_heads, head_dim, max_tokens, dtype, kv_format)
        self._views((batch, n_kv_heads, max_tokens, head_dim))

    def _views(self, shape):
        kp, vp = dkv_cache_host_ptrs(self.h)
        n = int(np.prod(shape))
        el = ctypes.c_uint16 if self.kv_format == "native" else ctypes.c_uint8
        self.k_host = np.ctypeslib.as_array((el * n).from_address(kp)).reshape(shape)
        self.v_host = np.ctypeslib.as_array((el * n).from_address(vp)).reshape(shape)

    def set_lengths(self, lens):
        dkv_cache_set_lengths(self.h, np.broadcast_to(np.asarray(lens, np.int32), (self.B,)))

    def lengths(self):
        return dkv_cache_get_lengths(self.h, self.B)

    def decode(self, x, wq, wk, wv, n_q_heads, out, stream=None):
        dkv_decode(self.h, x, wq, wk, wv, x.shape[-1], n_q_heads, out, stream)

    def prefill(self, x, wq, wk, wv, n_q_heads, out, stream=None):
        dkv_prefill(self.h, x, x.shape[1], wq, wk, wv, x.shape[-1], n_q_heads, out, stream)

    def sync(self, stream=None):
        dkv_sync_status(self.h, stream)

    def free(self):
        if self.h is not None:
            self.k_host = self.v_host = None
            dkv_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class PagedKVCache(KVCache):
    """A paged cache: numpy views of the K and V page pools
    ([num_pages, Hkv, page_tokens, D] uint16 each) and the page table.

    kv_format "e2m1": 4-bit pools ([num_pages, Hkv, page_tokens * D * 9 // 16] uint8) for
    ``append`` and ``attend``, whose lengths, page table and slots are device tensors
    (dkv_step_plan); ``k_pool`` and ``v_pool`` are the pools as pinned torch tensors.
    kv_format "e4m3_block": the same with E4M3 pools ([num_pages, Hkv, page_tokens, D]) and block scales, ``k_scales`` and
    ``v_scales`` ([num_pages, Hkv, page_tokens // 16] fp32), which are CUDA tensors: they are read with every block.
    ``pools`` are the tensors that dkv_pages_copy moves for a page of either."""

    def __init__(self, batch, n_kv_heads, head_dim, page_tokens, num_pages, max_pages_per_seq,
                 dtype="bf16", kv_format="native"):
        self.B, self.Hkv, self.D = batch, n_kv_heads, head_dim
        self.page_tokens, self.num_pages, self.max_pages = page_tokens, num_pages, max_pages_per_seq
        self.S_max = page_tokens * max_pages_per_seq
        self.dtype, self.kv_format = dtype, kv_format
        blocks = kv_format == "e4m3_block"
        if blocks and page_tokens % 16:
            raise ValueError(f"pages of {page_tokens} tokens: blocks are 16")
        # (the library's E4M3 cache without scales, whose projecting calls are refused here, has no fp16)
        self.h = dkv_cache_alloc_ex(batch, n_kv_heads, head_dim, 0, "bf16" if blocks else dtype,
                                    "e4m3" if blocks else kv_format, 1, page_tokens, num_pages, max_pages_per_seq)
        self.k_pool = self.v_pool = self.k_scales = self.v_scales = None
        if blocks or kv_format == "e2m1":
            import torch
            self._views((num_pages, n_kv_heads, page_tokens, head_dim) if blocks else
                        (num_pages, n_kv_heads, page_tokens * head_dim * 9 // 16))
            self.k_pool, self.v_pool = torch.from_numpy(self.k_host), torch.from_numpy(self.v_host)
            if blocks:
                self.k_scales, self.v_scales = (torch.ones((num_pages, n_kv_heads, page_tokens // 16), device="cuda")
                                                for _ in "kv")
        else:
            self._views((num_pages, n_kv_heads, page_tokens, head_dim))
        self.table = np.full((batch, max_pages_per_seq), -1, np.int32)

    def append(self, q, k, v, positions, slots, q_out, **more):
        """dkv_qkv_append into this E2M1 cache, dkv_block_append into one with block scales."""
        if self.k_scales is not None:
            dkv_block_append(q, k, v, positions, slots, self.k_pool, self.v_pool, self.k_scales, self.v_scales, q_out, **more)
        else:
            dkv_qkv_append(q, k, v, positions, slots, self.k_pool, self.v_pool, q_out, **more)

    def attend(self, q, page_table, kv_len, out, **more):
        """dkv_paged_attend over this E2M1 cache, dkv_block_attend over one with block scales."""
        if self.k_scales is not None:
            dkv_block_attend(q, self.k_pool, self.v_pool, self.k_scales, self.v_scales, page_table, kv_len, out, **more)
        else:
            dkv_paged_attend(q, self.k_pool, self.v_pool, page_table, kv_len, out, **more)

    @property
    def pools(self):
        """What a page of this cache consists of, for dkv_pages_copy."""
        return [t for t in (self.k_pool, self.v_pool, self.k_scales, self.v_scales) if t is not None]

    def decode(self, *args, **more):
        self._projects()
        super().decode(*args, **more)

    def prefill(self, *args, **more):
        self._projects()
        super().prefill(*args, **more)

    def _projects(self):
        if self.k_scales is not None:
            raise DkvError(2, "PagedKVCache", "a cache with block scales is served by append and attend")

    def free(self):
        self.k_pool = self.v_pool = self.k_scales = self.v_scales = None
        super().free()

    def set_page_table(self, table):
        dkv_cache_set_page_table(self.h, table)
        self.table = np.array(table, dtype=np.int32, copy=True)


class LayeredKVCache(KVCache):
    """A whole model's caches: numpy views [layers, B, Hkv, S_max, D] (uint16)
    of the pinned K and V, per-layer decode / prefill and the captured step."""

    def __init__(self, layers, batch, n_kv_heads, head_dim, max_tokens, dtype="bf16",
                 kv_format="native"):
        self.L, self.B, self.Hkv, self.D, self.S_max = layers, batch, n_kv_heads, head_dim, max_tokens
        self.dtype, self.kv_format = dtype, kv_format
        self.h = dkv_cache_alloc_ex(batch, n_kv_heads, head_dim, max_tokens, dtype, kv_format,
                                    layers)
        self._views((layers, batch, n_kv_heads, max_tokens, head_dim))

    def decode_layer(self, layer, x, wq, wk, wv, n_q_heads, out, stream=None):
        dkv_decode_layer(self.h, layer, x, wq, wk, wv, x.shape[-1], n_q_heads, out, stream)

    def prefill_layer(self, layer, x, wq, wk, wv, n_q_heads, out, stream=None):
        dkv_prefill_layer(self.h, layer, x, x.shape[1], wq, wk, wv, x.shape[-1], n_q_heads, out,
                          stream)

    def capture_step(self, xs, wqs, wks, wvs, n_q_heads, outs):
        dkv_step_graph_capture(self.h, xs[0].shape[-1], n_q_heads, xs, wqs, wks, wvs, outs)

    def launch_step(self, stream=None):
        dkv_step_graph_launch(self.h, stream)
