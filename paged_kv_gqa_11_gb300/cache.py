"""A paged K/V cache held in torch device memory, driven through libpa.

``PagedKVCache`` owns the allocator state (``Pool``), the device K and V
pools, a device error word and a reusable decode workspace.  Every operation is
one libpa call on the current CUDA stream; this module only allocates torch
buffers and passes pointers.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (PA_ERR_INVALID, PA_OK, PaError, Pool, load, load_calls, pa_append_rows, pa_append_rows_f16, pa_decode,
               pa_decode_workspace_size, pa_get_error)
from .rope import Rope


class PagedKVCache:
    def __init__(self, n_blocks: int, page_size: int, k_type: int, v_type: int | None = None,
                 n_kv_heads: int = 4, head_dim: int = 256, device: torch.device | str = "cuda",
                 k_pool: torch.Tensor | None = None, v_pool: torch.Tensor | None = None):
        """k_pool, v_pool: pools that exist already (uint8 on the cache's device, the pool's bytes, 16-byte aligned),
        else zeroed ones are made."""
        load()
        self.device = torch.device(device)
        self.pool = Pool(n_blocks, page_size, n_kv_heads, head_dim, k_type, v_type)
        self.page_size = page_size
        self.n_blocks = n_blocks
        self.n_kv_heads = n_kv_heads
        self.head_dim = head_dim
        self.k_type = k_type
        self.v_type = k_type if v_type is None else v_type
        self.k_pool = self._pool_buffer(k_pool, 0)
        self.v_pool = self._pool_buffer(v_pool, 1)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._ws = None
        self._ws_key = None

    def _pool_buffer(self, given: torch.Tensor | None, which: int) -> torch.Tensor:
        n = self.pool.bytes(which)
        if given is None:
            return torch.zeros(n, dtype=torch.uint8, device=self.device)
        if given.dtype != torch.uint8 or given.numel() != n or not given.is_contiguous():
            raise PaError(PA_ERR_INVALID, f"pool buffer: uint8, {n} bytes")
        # the calls pass its address on to kernels
        if not given.is_cuda or given.device.index != self._device_index() or given.data_ptr() % 16:
            raise PaError(PA_ERR_INVALID, f"pool buffer: on {self.device}, 16-byte aligned")
        return given

    def _device_index(self) -> int:
        return self.device.index if self.device.index is not None else torch.cuda.current_device()

    # ------------------------------------------------------------ append
    def append(self, k_rows: torch.Tensor, v_rows: torch.Tensor, row_seq: torch.Tensor, row_pos: torch.Tensor,
               block_table: torch.Tensor, stream=None) -> None:
        """Scatter packed rows [n][n_kv_heads][row_bytes] (device uint8) into the pools."""
        n = int(row_seq.shape[0])
        pa_append_rows(self.pool, self.k_pool, self.v_pool, k_rows, v_rows, row_seq, row_pos, n, block_table,
                       int(block_table.shape[1]), int(block_table.shape[0]), self.err, stream)

    def append_f16(self, k_rows: torch.Tensor, v_rows: torch.Tensor, row_seq: torch.Tensor, row_pos: torch.Tensor,
                   block_table: torch.Tensor, stream=None) -> None:
        """Quantise binary16 rows [n][n_kv_heads][head_dim] (device, float16 or their uint16
        bit patterns) into the pools' formats while scattering them."""
        n = int(row_seq.shape[0])
        pa_append_rows_f16(self.pool, self.k_pool, self.v_pool, k_rows, v_rows, row_seq, row_pos, n, block_table,
                           int(block_table.shape[1]), int(block_table.shape[0]), self.err, stream)

    def append_rope(self, rope: Rope, k: torch.Tensor, v: torch.Tensor, row_seq: torch.Tensor, row_pos: torch.Tensor,
                    block_table: torch.Tensor, k_weight: torch.Tensor | None = None, q: torch.Tensor | None = None,
                    q_weight: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                    q_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor | None:
        """Rows straight from a projection (stream, here and in read_rows and
        decode_prefix: as in Rope.apply): k and v [n][n_kv_heads][256], and if
        given q [n][heads][256] (parts of one tensor are fine).  Keys are
        normalised (with a weight), rotated to row_pos and stored, values stored;
        returns the queries, normalised and rotated, as q_dtype (default:
        q's own)."""
        return load_calls().append_rope(self.pool.address, self.n_kv_heads, self.k_pool, self.v_pool, rope.address, k, v,
                                       row_seq, row_pos, block_table, k_weight, q, q_weight, q_out, q_dtype, self.err,
                                       stream)

    # ------------------------------------------------------------ reading back
    def read_rows(self, row_seq: torch.Tensor, row_pos: torch.Tensor, block_table: torch.Tensor,
                  dtype: torch.dtype = torch.float16, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None, stream=None):
        """The cache's rows at (row_seq, row_pos) as values [n][n_kv_heads][256];
        returns (k, v).  With only one of k_out, v_out given, only that one is
        read."""
        return load_calls().read_rows(self.pool.address, self.n_kv_heads, self.k_pool, self.v_pool, row_seq, row_pos,
                                     block_table, dtype, k_out, v_out, self.err, stream)

    # ------------------------------------------------------------ moving
    def move_rows(self, src_seq: torch.Tensor, src_pos: torch.Tensor, dst_seq: torch.Tensor, dst_pos: torch.Tensor,
                  block_table: torch.Tensor, dst_table: torch.Tensor | None = None, rope: Rope | None = None,
                  rope_from: Rope | None = None, disjoint: bool = False, workspace: torch.Tensor | None = None, stream=None) -> None:
        """Rows (src_seq, src_pos) moved to (dst_seq, dst_pos), int32 [n] each, through
        block_table (the destinations through dst_table, if given).  All rows are
        read before any is written; disjoint: no row's destination is another's
        source (the caller's word; a launch less).  With a rope, keys are turned from
        their old position's angles (under rope_from, or rope) to the new one's
        and stored anew; without one, rows keep their bytes.  Workspace and
        stream: as decode_prefix."""
        load_calls().move_rows(self.pool.address, self.k_pool, self.v_pool, rope.address if rope is not None else 0,
                               rope_from.address if rope_from is not None else 0, src_seq, src_pos, dst_seq, dst_pos, block_table,
                               dst_table, disjoint, workspace, self.err, stream)

    def move_blocks(self, src: torch.Tensor, dst: torch.Tensor, block_table: torch.Tensor | None = None,
                    table_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Whole blocks src[i] copied to dst[i] (int32 [n]; none in both; src ascending if
        there is a table), and the table with dst[i] for every src[i] (into table_out, which
        may be the table, or a new tensor), which is returned: the device half of
        Pool.compact."""
        return load_calls().move_blocks(self.pool.address, self.k_pool, self.v_pool, src, dst, block_table, table_out, self.err, stream)

    # ------------------------------------------------------------ decode
    def workspace(self, n_seq: int, n_qtok: int) -> torch.Tensor:
        dev = self._device_index()
        key = (n_seq, n_qtok, dev)
        if self._ws is None or self._ws_key != key:
            nbytes = pa_decode_workspace_size(self.pool, n_seq, n_qtok, dev)
            if nbytes == 0:
                raise PaError(1, "pa_decode_workspace_size")
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self._ws_key = key
        return self._ws

    def decode(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens_dev: torch.Tensor,
               seq_lens_host: np.ndarray, n_qtok: int, scale: float = 1.0 / 16.0, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, want_lse: bool = True, stream=None, passes: str = "all"):
        """q: device fp32 [n_seq][n_qtok][n_q_heads][head_dim]; returns (out, lse)."""
        n_seq, _, hq, d = q.shape
        if out is None:
            out = torch.empty((n_seq, n_qtok, hq, d), dtype=torch.float32, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((n_seq, n_qtok, hq), dtype=torch.float32, device=self.device)
        sl = np.ascontiguousarray(seq_lens_host, dtype=np.int32)
        ws = self.workspace(n_seq, n_qtok)
        pa_decode(self.pool, q, self.k_pool, self.v_pool, block_table, int(block_table.shape[1]), seq_lens_dev, sl,
                  n_seq, n_qtok, hq, scale, out, lse, ws, ws.numel(), self.err, stream, passes=passes)
        return out, lse

    def decode_prefix(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens_dev: torch.Tensor,
                      seq_lens_host: np.ndarray, group_sizes, prefix_lens, n_qtok: int, scale: float = 1.0 / 16.0,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None, want_lse: bool = True,
                      workspace: torch.Tensor | None = None, stream=None):
        """decode for sequences that share prefixes: the batch is runs of
        group_sizes[g] sequences, whose first prefix_lens[g] positions hold the
        same rows; those are read once for the run.  q: [n_seq][n_qtok][heads][256]
        fp32, binary16 or bfloat16; out: q's shape, of q's type unless given;
        seq_lens_host, group_sizes, prefix_lens: host arrays of 32-bit whole
        numbers (numpy).
        Queries and keys are rounded to binary16 (decode keeps quantised keys
        exact): a logit is off by 2^-11 |q| |k| scale at most for each, so decode
        is the call for logits of hundreds.  A query value of fp32 or bfloat16
        past 65504 makes its row NaN, a stored V value past 65504 is infinite.
        The workspace is taken from torch's allocator for each call, so calls on
        several streams, and captured ones, each have their own.  Returns
        (out, lse)."""
        return load_calls().decode_prefix(self.pool.address, q, self.k_pool, self.v_pool, block_table, seq_lens_dev,
                                         seq_lens_host, group_sizes, prefix_lens, n_qtok, scale, out, lse, want_lse,
                                         workspace, self.err, stream)

    # ------------------------------------------------------------ attention over a window
    def attend_window(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens_dev: torch.Tensor, seq_lens_host: np.ndarray,
                      n_new, window: int = 0, sinks: int = 0, scale: float = 1.0 / 16.0, out: torch.Tensor | None = None,
                      lse: torch.Tensor | None = None, want_lse: bool = True, workspace: torch.Tensor | None = None, stream=None):
        """Causal attention of each sequence's newest n_new[s] tokens (0, 1, a
        few, a whole prompt), which are in the cache already: the token at
        position p sees the `window` keys up to its own (0: all) and the first
        `sinks`.  q: rows [tokens][heads][256] of fp32, binary16 or bfloat16, one
        sequence's after the other's (a part of a projection is fine); out: q's
        shape, of q's type unless given.  seq_lens_host, n_new: host arrays of
        32-bit whole numbers (numpy).  Pages that no new token sees are not read;
        they may have been released.  Rows of q after the last sequence's are left
        alone: those of a given out and lse stay, those of new ones are zeros.
        Precision, workspace and streams: as decode_prefix (keys, values and
        weights rounded to binary16 whatever out's type is; how, also depends on
        the batch).  For single tokens that see long contexts whole, decode is
        exacter and faster.  Returns (out, lse)."""
        return load_calls().attend_window(self.pool.address, q, self.k_pool, self.v_pool, block_table, seq_lens_dev,
                                          seq_lens_host, n_new, window, sinks, scale, out, lse, want_lse, workspace, self.err,
                                          stream)

    def check(self, stream=None) -> int:
        """Synchronise, read and reset the device error word."""
        return pa_get_error(self.err, stream)

    def raise_on_error(self, stream=None) -> None:
        rc = self.check(stream)
        if rc != PA_OK:
            raise PaError(rc, "device")
