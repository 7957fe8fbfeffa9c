"""Norm and position rotation of query and key heads (``pa_norm_rope``).

``Rope`` holds what a model fixes once -- frequencies, pairing, norm constants
-- and is passed to the calls that rotate: ``Rope.apply`` for query and key
heads that stay outside a cache, ``PagedKVCache.append_rope`` for rows on their
way into one.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import PaError, PA_ERR_INVALID, RopeDesc, dtype_number, pa_norm_rope

HEAD_DIM = 256


def heads_of(x: torch.Tensor | None, what: str) -> tuple[int, int]:
    """(row stride in elements, heads) of rows [n][heads][256] whose heads are packed; (0, 0) for None."""
    if x is None:
        return 0, 0
    n, h, d = x.shape
    s = x.stride()
    if d != HEAD_DIM or s[2] != 1 or (h > 1 and s[1] != HEAD_DIM):
        raise PaError(PA_ERR_INVALID, f"{what}: rows of packed heads of {HEAD_DIM} values")
    return (s[0] if n > 1 else max(s[0], h * HEAD_DIM)), h


class Rope:
    def __init__(self, inv_freq, interleaved: bool = False, eps: float = 1e-6, weight_offset: float = 0.0,
                 attn_factor: float = 1.0):
        """inv_freq: radians per position of each rotated pair (a sequence of
        floats; 2 * len of them is the rotated width, a multiple of 16)."""
        f = [float(x) for x in inv_freq]
        if len(f) > 128:
            raise PaError(PA_ERR_INVALID, "Rope: at most 128 pairs")
        self.desc = RopeDesc(2 * len(f), int(bool(interleaved)), eps, weight_offset, attn_factor,
                             (C.c_double * 128)(*f))
        self.address = C.addressof(self.desc)

    @classmethod
    def from_theta(cls, rot_dim: int, theta: float, **kw) -> "Rope":
        """The usual frequencies theta^(-2 i / rot_dim)."""
        return cls([float(theta) ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], **kw)

    def apply(self, q: torch.Tensor | None, k: torch.Tensor | None, row_pos: torch.Tensor,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
              out_dtype: torch.dtype | None = None, stream=None):
        """q [n][heads][256] and k [n][kv heads][256] (either may be None; parts
        of one projection are fine), normalised where a weight is given and
        rotated to row_pos (int32 [n]).  Returns (q_out, k_out); an output may be
        its input."""
        some = q if q is not None else k
        if some is None:
            raise PaError(PA_ERR_INVALID, "Rope.apply: q or k")
        n = some.shape[0]
        in_type = dtype_number(some.dtype)
        if q is not None and k is not None and (k.dtype != q.dtype or k.shape[0] != n):
            raise PaError(PA_ERR_INVALID, "Rope.apply: q and k of one type and row count")
        for given in (q_out, k_out):
            if given is not None:
                out_dtype = given.dtype if out_dtype is None else out_dtype
                if given.dtype != out_dtype:
                    raise PaError(PA_ERR_INVALID, "Rope.apply: outputs of one type")
        out_dtype = some.dtype if out_dtype is None else out_dtype
        w_type = weight_type(q_weight, k_weight)
        check_index(row_pos, n, "row_pos")
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=out_dtype, device=k.device)
        for a, b in ((q, q_out), (k, k_out)):
            if (a is None) != (b is None) or (a is not None and a.shape != b.shape):
                raise PaError(PA_ERR_INVALID, "Rope.apply: outputs of the inputs' shape")
        qs, hq = heads_of(q, "q")
        ks, hk = heads_of(k, "k")
        pa_norm_rope(self.address, q, qs, hq, k, ks, hk, in_type, q_weight, k_weight, w_type, row_pos, n, q_out,
                     heads_of(q_out, "q_out")[0], k_out, heads_of(k_out, "k_out")[0], dtype_number(out_dtype), stream)
        return q_out, k_out


def weight_type(*weights) -> int:
    """The number of the weights' one type (any, if there is none)."""
    t = None
    for w in weights:
        if w is None:
            continue
        if w.shape != (HEAD_DIM,) or not w.is_contiguous() or (t is not None and w.dtype != t):
            raise PaError(PA_ERR_INVALID, f"weights: [{HEAD_DIM}], of one type")
        t = w.dtype
    return dtype_number(torch.float32 if t is None else t)


def check_index(x: torch.Tensor, n: int, what: str) -> None:
    if x.dtype != torch.int32 or x.dim() != 1 or x.shape[0] != n or not x.is_contiguous():
        raise PaError(PA_ERR_INVALID, f"{what}: int32 [{n}]")


def check_table(table: torch.Tensor) -> None:
    if table.dtype != torch.int32 or table.dim() != 2 or not table.is_contiguous():
        raise PaError(PA_ERR_INVALID, "block_table: int32 [n_seq][pages], contiguous")
