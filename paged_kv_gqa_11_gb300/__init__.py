"""Paged GQA decode attention on GB300: Python binding of libpa.

A thin ctypes layer over the C ABI declared in ``include/pa.h``: it marshals
pointers, sizes and the current CUDA stream and returns status codes.  All the
work -- allocation bookkeeping, the append scatter, the split decode and its
merge -- runs inside libpa (host C++ and sm_103a CUDA kernels).  There is no
Python or CPU fallback: if libpa has not been built, every call raises.

Device buffers are torch tensors (torch owns the memory); the library never
allocates device memory.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

from . import _build

__all__ = [
    "PA_F16", "PA_Q4_0", "PA_Q8_0", "PaError", "Pool", "load", "load_calls", "row_bytes", "pa_append_rows", "pa_append_rows_f16", "pa_copy_blocks", "pa_decode",
    "pa_decode_workspace_size", "pa_decode_plan", "pa_get_error", "pa_selftest_wait_timeout", "status_name",
    "library_path", "pa_decode_noalloc", "PA_DT_F32", "PA_DT_F16", "PA_DT_BF16", "RopeDesc", "dtype_number",
    "pa_norm_rope", "pa_append_rows_rope", "pa_read_rows", "pa_decode_prefix", "pa_decode_prefix_workspace_size",
    "pa_attend_window", "pa_attend_window_workspace_size", "pa_move_rows", "pa_move_rows_workspace_size", "pa_move_blocks",
]

PA_F16, PA_Q4_0, PA_Q8_0 = 1, 2, 8
PA_DT_F32, PA_DT_F16, PA_DT_BF16 = 0, 1, 30
STATUS = ["PA_OK", "PA_ERR_INVALID", "PA_ERR_UNSUPPORTED", "PA_ERR_OOM", "PA_ERR_STALE", "PA_ERR_BOUNDS",
          "PA_ERR_TIMEOUT", "PA_ERR_CUDA"]
PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_OOM, PA_ERR_STALE, PA_ERR_BOUNDS, PA_ERR_TIMEOUT, PA_ERR_CUDA = range(8)

# Every entry point declared in include/pa.h.
EXPORTS = ["pa_pool_create", "pa_pool_destroy", "pa_pool_get_desc", "pa_row_bytes", "pa_pool_bytes",
           "pa_alloc_blocks", "pa_release", "pa_block_index", "pa_pool_free_count", "pa_share_blocks", "pa_block_refcount",
           "pa_cow_blocks", "pa_copy_blocks", "pa_append_rows", "pa_append_rows_f16",
           "pa_decode", "pa_decode_split", "pa_decode_merge", "pa_decode_workspace_size", "pa_decode_plan", "pa_get_error", "pa_status_string",
           "pa_selftest_wait_timeout", "pa_decode_noalloc", "pa_norm_rope", "pa_append_rows_rope", "pa_read_rows",
           "pa_decode_prefix", "pa_decode_prefix_workspace_size", "pa_attend_window", "pa_attend_window_workspace_size",
           "pa_compact_blocks", "pa_move_blocks", "pa_move_rows", "pa_move_rows_workspace_size"]


class PaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_name(status)}" if what else status_name(status))


def status_name(s: int) -> str:
    return STATUS[s] if 0 <= s < len(STATUS) else f"PA_STATUS_{s}"


class PoolDesc(C.Structure):
    _fields_ = [("n_blocks", C.c_uint32), ("page_size", C.c_uint32), ("n_kv_heads", C.c_uint32),
                ("head_dim", C.c_uint32), ("k_type", C.c_int32), ("v_type", C.c_int32)]


class RopeDesc(C.Structure):
    _fields_ = [("rot_dim", C.c_uint32), ("interleaved", C.c_int32), ("eps", C.c_float),
                ("weight_offset", C.c_float), ("attn_factor", C.c_float), ("inv_freq", C.c_double * 128)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load():
    """Load libpa.so; raises if it has not been built (no fallback)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"libpa is not built ({path} missing); run paged_kv_gqa_11_gb300._build.build()")
        L = C.CDLL(path)
        vp, u32, i32, sz, i64 = C.c_void_p, C.c_uint32, C.c_int32, C.c_size_t, C.c_int64
        sig = {
            "pa_pool_create": (C.c_int, [C.POINTER(PoolDesc), C.POINTER(vp)]),
            "pa_pool_destroy": (None, [vp]),
            "pa_pool_get_desc": (C.c_int, [vp, C.POINTER(PoolDesc)]),
            "pa_row_bytes": (sz, [i32, u32]),
            "pa_pool_bytes": (sz, [vp, C.c_int]),
            "pa_alloc_blocks": (C.c_int, [vp, u32, vp]),
            "pa_release": (C.c_int, [vp, vp, u32]),
            "pa_block_index": (C.c_int, [vp, C.c_uint64, C.POINTER(i32)]),
            "pa_pool_free_count": (u32, [vp]),
            "pa_share_blocks": (C.c_int, [vp, vp, u32]),
            "pa_block_refcount": (C.c_int, [vp, C.c_uint64, C.POINTER(u32)]),
            "pa_cow_blocks": (C.c_int, [vp, vp, u32, vp, vp, vp, C.POINTER(u32)]),
            "pa_copy_blocks": (C.c_int, [vp, vp, vp, vp, vp, u32, vp, vp]),
            "pa_append_rows": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, u32, vp, u32, u32, vp, vp]),
            "pa_append_rows_f16": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, u32, vp, u32, u32, vp, vp]),
            "pa_decode": (C.c_int, [vp, vp, vp, vp, vp, u32, vp, vp, u32, u32, u32, C.c_float, vp, vp, vp, sz,
                                    vp, vp]),
            "pa_decode_workspace_size": (sz, [vp, u32, u32, C.c_int]),
            "pa_decode_plan": (C.c_int, [vp, vp, u32, u32, C.c_int, C.POINTER(u32), C.POINTER(u32),
                                         C.POINTER(u32), C.POINTER(u32)]),
            "pa_get_error": (C.c_int, [vp, vp]),
            "pa_status_string": (C.c_char_p, [C.c_int]),
            "pa_selftest_wait_timeout": (C.c_int, [u32, vp, vp]),
            "pa_decode_noalloc": (C.c_int, [vp, vp, vp, vp, vp, u32, vp, vp, u32, u32, u32, C.c_float, vp, vp,
                                            vp, vp]),
            "pa_norm_rope": (C.c_int, [vp, vp, i64, u32, vp, i64, u32, i32, vp, vp, i32, vp, u32, vp, i64, vp, i64, i32,
                                       vp]),
            "pa_append_rows_rope": (C.c_int, [vp, vp, vp, vp, vp, i64, vp, i64, i32, vp, i32, vp, i64, u32, vp, vp, i64,
                                              i32, vp, vp, u32, vp, u32, u32, vp, vp]),
            "pa_read_rows": (C.c_int, [vp, vp, vp, vp, vp, u32, vp, u32, u32, vp, vp, i32, vp, vp]),
            "pa_decode_prefix": (C.c_int, [vp, vp, i32, vp, vp, vp, u32, vp, vp, u32, vp, vp, u32, u32, u32, C.c_float,
                                           vp, i32, vp, vp, sz, vp, vp]),
            "pa_decode_prefix_workspace_size": (sz, [vp, u32, u32, u32, C.c_int]),
            "pa_attend_window": (C.c_int, [vp, vp, i64, i32, vp, vp, vp, u32, vp, vp, vp, u32, u32, u32, u32, C.c_float, vp,
                                           i64, i32, vp, vp, sz, vp, vp]),
            "pa_attend_window_workspace_size": (sz, [vp, vp, vp, u32, u32, u32, C.c_int]),
            "pa_compact_blocks": (C.c_int, [vp, u32, vp, vp, C.POINTER(u32)]),
            "pa_move_blocks": (C.c_int, [vp, vp, vp, vp, vp, u32, vp, vp, C.c_uint64, vp, vp]),
            "pa_move_rows": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, u32, vp, u32, u32, vp, u32, u32, i32, vp, sz, vp, vp]),
            "pa_move_rows_workspace_size": (sz, [vp, u32]),
        }
        sig["pa_decode_split"] = sig["pa_decode_merge"] = sig["pa_decode"]
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
        return L


_calls = None


def load_calls():
    """The Python module over the calls that run once per layer and step
    (csrc/pa_calls.cpp); raises if it has not been built (no fallback)."""
    global _calls
    if _calls is not None:
        return _calls
    load()
    with _lock:
        if _calls is None:
            import importlib.machinery
            import importlib.util

            import torch  # noqa: F401  (its libraries, before the module that uses them)
            path = _build.CALLS_PATH
            if not os.path.exists(path):
                raise RuntimeError(f"pa_calls is not built ({path} missing); run paged_kv_gqa_11_gb300._build.build()")
            loader = importlib.machinery.ExtensionFileLoader("pa_calls", path)
            m = importlib.util.module_from_spec(importlib.util.spec_from_loader("pa_calls", loader))
            loader.exec_module(m)
            m.set_error(PaError)
            _calls = m
        return _calls


def row_bytes(t: int, head_dim: int = 256) -> int:
    return int(load().pa_row_bytes(t, head_dim))


def _ptr(x) -> int | None:
    """Device/host address of a torch tensor, an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):  # numpy array
        return x.ctypes.data
    raise TypeError(type(x))


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, what: str) -> None:
    if rc != PA_OK:
        raise PaError(rc, what)


class Pool:
    """Allocator state of one K/V pool (host metadata; see pa_pool_create)."""

    def __init__(self, n_blocks: int, page_size: int, n_kv_heads: int = 4, head_dim: int = 256,
                 k_type: int = PA_F16, v_type: int | None = None):
        L = load()
        self.desc = PoolDesc(n_blocks, page_size, n_kv_heads, head_dim, k_type,
                             k_type if v_type is None else v_type)
        h = C.c_void_p()
        _check(L.pa_pool_create(C.byref(self.desc), C.byref(h)), "pa_pool_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    @property
    def address(self) -> int:
        return self._h.value

    def close(self):
        if getattr(self, "_h", None):
            load().pa_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def bytes(self, which: int) -> int:
        return int(load().pa_pool_bytes(self._h, which))

    def alloc(self, n: int) -> list[int]:
        buf = (C.c_uint64 * max(n, 1))()
        _check(load().pa_alloc_blocks(self._h, n, buf), "pa_alloc_blocks")
        return list(buf[:n])

    def alloc_status(self, n: int):
        buf = (C.c_uint64 * max(n, 1))()
        rc = load().pa_alloc_blocks(self._h, n, buf)
        return rc, (list(buf[:n]) if rc == PA_OK else [])

    def release(self, handles) -> int:
        arr = (C.c_uint64 * max(len(handles), 1))(*handles)
        return int(load().pa_release(self._h, arr, len(handles)))

    def block_index(self, handle: int):
        idx = C.c_int32(-1)
        rc = load().pa_block_index(self._h, handle, C.byref(idx))
        return rc, idx.value

    def free_count(self) -> int:
        return int(load().pa_pool_free_count(self._h))

    def share(self, handles) -> int:
        arr = (C.c_uint64 * max(len(handles), 1))(*handles)
        return int(load().pa_share_blocks(self._h, arr, len(handles)))

    def refcount(self, handle: int):
        n = C.c_uint32(0)
        rc = load().pa_block_refcount(self._h, handle, C.byref(n))
        return rc, n.value

    def cow(self, handles):
        """Returns (status, handles to write through, [(src index, dst index)] copies)."""
        k = max(len(handles), 1)
        arr = (C.c_uint64 * k)(*handles)
        out = (C.c_uint64 * k)()
        src, dst = (C.c_int32 * k)(), (C.c_int32 * k)()
        nc = C.c_uint32(0)
        rc = int(load().pa_cow_blocks(self._h, arr, len(handles), out, src, dst, C.byref(nc)))
        if rc != PA_OK:
            return rc, [], []
        return rc, list(out[:len(handles)]), [(src[i], dst[i]) for i in range(nc.value)]


    def compact(self) -> list[tuple[int, int]]:
        """Brings the live blocks to the front; returns the moved blocks' (old handle, new handle), ascending by
        the old index.  The caller then moves their rows (pa_move_blocks, by the handles' low 32 bits) and
        puts the new handles in the old ones' place."""
        n = C.c_uint32(0)
        while True:
            k = n.value
            old, new = (C.c_uint64 * max(k, 1))(), (C.c_uint64 * max(k, 1))()
            rc = int(load().pa_compact_blocks(self._h, k, old, new, C.byref(n)))
            if rc == PA_OK:
                return list(zip(old[:n.value], new[:n.value]))
            if n.value <= k:  # not for the arrays' size
                raise PaError(rc, "pa_compact_blocks")


def pa_append_rows(pool: Pool, k_pool, v_pool, k_rows, v_rows, row_seq, row_pos, n_rows: int, block_table,
                   table_stride: int, n_seq: int, err, stream=None) -> None:
    rc = load().pa_append_rows(pool.handle, _ptr(k_pool), _ptr(v_pool), _ptr(k_rows), _ptr(v_rows), _ptr(row_seq),
                               _ptr(row_pos), n_rows, _ptr(block_table), table_stride, n_seq, _ptr(err),
                               _stream(stream))
    _check(rc, "pa_append_rows")


def pa_append_rows_f16(pool: Pool, k_pool, v_pool, k_rows, v_rows, row_seq, row_pos, n_rows: int, block_table,
                       table_stride: int, n_seq: int, err, stream=None) -> None:
    """Rows as binary16 [n_rows][n_kv_heads][head_dim], quantised into the pool's formats."""
    rc = load().pa_append_rows_f16(pool.handle, _ptr(k_pool), _ptr(v_pool), _ptr(k_rows), _ptr(v_rows),
                                   _ptr(row_seq), _ptr(row_pos), n_rows, _ptr(block_table), table_stride, n_seq,
                                   _ptr(err), _stream(stream))
    _check(rc, "pa_append_rows_f16")


def pa_copy_blocks(pool: Pool, k_pool, v_pool, src, dst, n: int, err, stream=None) -> None:
    """Copy whole blocks src[i] -> dst[i] (device int32 arrays) in both pools."""
    rc = load().pa_copy_blocks(pool.handle, _ptr(k_pool), _ptr(v_pool), _ptr(src), _ptr(dst), n, _ptr(err),
                               _stream(stream))
    _check(rc, "pa_copy_blocks")


def pa_decode_workspace_size(pool: Pool, n_seq: int, n_qtok: int, device: int = 0) -> int:
    return int(load().pa_decode_workspace_size(pool.handle, n_seq, n_qtok, device))


def pa_decode_plan(pool: Pool, seq_lens_host, n_qtok: int, device: int = 0) -> dict:
    import numpy as np
    sl = np.ascontiguousarray(seq_lens_host, dtype=np.int32)
    a, b, c, d = C.c_uint32(), C.c_uint32(), C.c_uint32(), C.c_uint32()
    _check(load().pa_decode_plan(pool.handle, sl.ctypes.data, len(sl), n_qtok, device, C.byref(a), C.byref(b),
                                 C.byref(c), C.byref(d)), "pa_decode_plan")
    return {"ctas": a.value, "tiles": b.value, "tile_keys": c.value, "partials": d.value}


def pa_decode(pool: Pool, q, k_pool, v_pool, block_table, table_stride: int, seq_lens_dev, seq_lens_host,
              n_seq: int, n_qtok: int, n_q_heads: int, scale: float, out, lse, workspace, ws_bytes: int, err,
              stream=None, check: bool = True, passes: str = "all") -> int:
    """seq_lens_host: a host int32 buffer (numpy array or address) that stays
    alive for the call.  passes: "all" (pa_decode), "split" (pa_decode_split)
    or "merge" (pa_decode_merge)."""
    fn = {"all": "pa_decode", "split": "pa_decode_split", "merge": "pa_decode_merge"}[passes]
    rc = getattr(load(), fn)(pool.handle, _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), table_stride,
                          _ptr(seq_lens_dev), _ptr(seq_lens_host), n_seq, n_qtok, n_q_heads, C.c_float(scale),
                          _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(err), _stream(stream))
    if check:
        _check(rc, "pa_decode")
    return rc


def pa_get_error(err, stream=None) -> int:
    return int(load().pa_get_error(_ptr(err), _stream(stream)))


def pa_selftest_wait_timeout(timeout_us: int, err, stream=None) -> int:
    return int(load().pa_selftest_wait_timeout(timeout_us, _ptr(err), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def pa_decode_noalloc(pool: Pool, q, k_pool, v_pool, block_table, table_stride: int, seq_lens_dev, seq_lens_host,
                      n_seq: int, n_qtok: int, n_q_heads: int, scale: float, out, lse, err, stream=None) -> int:
    """pa_decode with the library's fixed scratch instead of a caller workspace
    (for callers that cannot allocate device memory); returns the status."""
    return int(load().pa_decode_noalloc(pool.handle, _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                        table_stride, _ptr(seq_lens_dev), _ptr(seq_lens_host), n_seq, n_qtok,
                                        n_q_heads, C.c_float(scale), _ptr(out), _ptr(lse), _ptr(err),
                                        _stream(stream)))


_DTYPES = {}


def dtype_number(t) -> int:
    """The library's number of a torch dtype (float32, float16, bfloat16)."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: PA_DT_F32, torch.float16: PA_DT_F16, torch.bfloat16: PA_DT_BF16})
    if t not in _DTYPES:
        raise PaError(PA_ERR_UNSUPPORTED, str(t))
    return _DTYPES[t]


def pa_norm_rope(rope: int, q, q_stride: int, n_q_heads: int, k, k_stride: int, n_kv_heads: int, in_type: int,
                 q_weight, k_weight, w_type: int, row_pos, n_rows: int, q_out, q_out_stride: int, k_out,
                 k_out_stride: int, out_type: int, stream=None) -> None:
    """rope: the address of a RopeDesc; strides in elements between rows."""
    _check(load().pa_norm_rope(rope, _ptr(q), q_stride, n_q_heads, _ptr(k), k_stride, n_kv_heads, in_type,
                               _ptr(q_weight), _ptr(k_weight), w_type, _ptr(row_pos), n_rows, _ptr(q_out),
                               q_out_stride, _ptr(k_out), k_out_stride, out_type, _stream(stream)), "pa_norm_rope")


def pa_append_rows_rope(pool: Pool, k_pool, v_pool, rope: int, k_rows, k_stride: int, v_rows, v_stride: int,
                        in_type: int, k_weight, w_type: int, q, q_stride: int, n_q_heads: int, q_weight, q_out,
                        q_out_stride: int, q_out_type: int, row_seq, row_pos, n_rows: int, block_table,
                        table_stride: int, n_seq: int, err, stream=None) -> None:
    """Keys normalised, rotated and stored, values stored, queries normalised and rotated (q may be None)."""
    _check(load().pa_append_rows_rope(pool.handle, _ptr(k_pool), _ptr(v_pool), rope, _ptr(k_rows), k_stride,
                                      _ptr(v_rows), v_stride, in_type, _ptr(k_weight), w_type, _ptr(q), q_stride,
                                      n_q_heads, _ptr(q_weight), _ptr(q_out), q_out_stride, q_out_type, _ptr(row_seq),
                                      _ptr(row_pos), n_rows, _ptr(block_table), table_stride, n_seq, _ptr(err),
                                      _stream(stream)), "pa_append_rows_rope")


def pa_read_rows(pool: Pool, k_pool, v_pool, row_seq, row_pos, n_rows: int, block_table, table_stride: int,
                 n_seq: int, k_out, v_out, out_type: int, err, stream=None) -> None:
    """Rows [n_rows][n_kv_heads][head_dim] of the pools as values of out_type (k_out or v_out may be None)."""
    _check(load().pa_read_rows(pool.handle, _ptr(k_pool), _ptr(v_pool), _ptr(row_seq), _ptr(row_pos), n_rows,
                               _ptr(block_table), table_stride, n_seq, _ptr(k_out), _ptr(v_out), out_type, _ptr(err),
                               _stream(stream)), "pa_read_rows")


def pa_decode_prefix_workspace_size(pool: Pool, n_seq: int, n_groups: int, n_qtok: int, device: int = 0) -> int:
    return int(load().pa_decode_prefix_workspace_size(pool.handle, n_seq, n_groups, n_qtok, device))


def pa_decode_prefix(pool: Pool, q, q_type: int, k_pool, v_pool, block_table, table_stride: int, seq_lens_dev,
                     seq_lens_host, n_seq: int, group_sizes, prefix_lens, n_groups: int, n_qtok: int, n_q_heads: int,
                     scale: float, out, out_type: int, lse, workspace, ws_bytes: int, err, stream=None,
                     check: bool = True) -> int:
    """seq_lens_host (int32), group_sizes (uint32) and prefix_lens (int32): host
    buffers that stay alive for the call."""
    rc = load().pa_decode_prefix(pool.handle, _ptr(q), q_type, _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                 table_stride, _ptr(seq_lens_dev), _ptr(seq_lens_host), n_seq, _ptr(group_sizes),
                                 _ptr(prefix_lens), n_groups, n_qtok, n_q_heads, scale, _ptr(out), out_type, _ptr(lse),
                                 _ptr(workspace), ws_bytes, _ptr(err), _stream(stream))
    if check:
        _check(rc, "pa_decode_prefix")
    return rc


def pa_attend_window_workspace_size(pool: Pool, seq_lens_host, n_new, window: int = 0, sinks: int = 0, device: int = 0) -> int:
    import numpy as np
    sl, nn = (np.ascontiguousarray(x, dtype=np.int32) for x in (seq_lens_host, n_new))
    if sl.ndim != 1 or sl.shape != nn.shape:
        raise PaError(PA_ERR_INVALID, "a length and a number of new tokens per sequence")
    return int(load().pa_attend_window_workspace_size(pool.handle, sl.ctypes.data, nn.ctypes.data, len(sl), window, sinks, device))


def pa_attend_window(pool: Pool, q, q_stride: int, q_type: int, k_pool, v_pool, block_table, table_stride: int, seq_lens_dev,
                     seq_lens_host, n_new, n_seq: int, n_q_heads: int, window: int, sinks: int, scale: float, out,
                     out_stride: int, out_type: int, lse, workspace, ws_bytes: int, err, stream=None, check: bool = True) -> int:
    """seq_lens_host, n_new: host int32 buffers that stay alive for the call; strides in elements between rows."""
    rc = load().pa_attend_window(pool.handle, _ptr(q), q_stride, q_type, _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                 table_stride, _ptr(seq_lens_dev), _ptr(seq_lens_host), _ptr(n_new), n_seq, n_q_heads, window,
                                 sinks, scale, _ptr(out), out_stride, out_type, _ptr(lse), _ptr(workspace), ws_bytes, _ptr(err),
                                 _stream(stream))
    if check:
        _check(rc, "pa_attend_window")
    return rc


def pa_move_blocks(pool: Pool, k_pool, v_pool, src, dst, n: int, table, table_out, n_entries: int, err, stream=None) -> None:
    """Copy whole blocks src[i] -> dst[i] in both pools and write tables with the new indices (src ascending)."""
    _check(load().pa_move_blocks(pool.handle, _ptr(k_pool), _ptr(v_pool), _ptr(src), _ptr(dst), n, _ptr(table),
                                 _ptr(table_out), n_entries, _ptr(err), _stream(stream)), "pa_move_blocks")


def pa_move_rows_workspace_size(pool: Pool, n_rows: int) -> int:
    return int(load().pa_move_rows_workspace_size(pool.handle, n_rows))


def pa_move_rows(pool: Pool, k_pool, v_pool, rope: int | None, rope_from: int | None, src_seq, src_pos, dst_seq, dst_pos,
                 n_rows: int, src_table, src_stride: int, src_n_seq: int, dst_table, dst_stride: int, dst_n_seq: int,
                 disjoint: bool, workspace, ws_bytes: int, err, stream=None) -> None:
    """Rows moved to other places, keys turned to them (rope, rope_from: addresses of RopeDescs, or None)."""
    _check(load().pa_move_rows(pool.handle, _ptr(k_pool), _ptr(v_pool), rope, rope_from, _ptr(src_seq), _ptr(src_pos),
                               _ptr(dst_seq), _ptr(dst_pos), n_rows, _ptr(src_table), src_stride, src_n_seq,
                               _ptr(dst_table), dst_stride, dst_n_seq, int(disjoint), _ptr(workspace), ws_bytes, _ptr(err),
                               _stream(stream)), "pa_move_rows")
