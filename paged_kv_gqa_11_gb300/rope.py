"""Norm and position rotation of query and key heads (``pa_norm_rope``).

``Rope`` holds what a model fixes once -- frequencies, pairing, norm constants
-- and is passed to the calls that rotate: ``Rope.apply`` for query and key
heads that stay outside a cache, ``PagedKVCache.append_rope`` for rows on their
way into one.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import PA_ERR_INVALID, PaError, RopeDesc, load_calls


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

    @property
    def address(self) -> int:
        """Of the constants, as the calls take them: in a copy, of the copy's own."""
        return C.addressof(self.desc)

    @classmethod
    def from_theta(cls, rot_dim: int, theta: float, **kw) -> "Rope":
        """The usual frequencies theta^(-2 i / rot_dim); rot_dim is even, 0 to 256."""
        if rot_dim % 2 or not 0 <= rot_dim <= 256:
            raise PaError(PA_ERR_INVALID, "Rope: rot_dim is even, 0 to 256")
        return cls([float(theta) ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], **kw)

    def apply(self, q: torch.Tensor | None, k: torch.Tensor | None, row_pos: torch.Tensor,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
              out_dtype: torch.dtype | None = None, stream=None):
        """q [n][heads][256] and k [n][kv heads][256] (either may be None; parts
        of one projection are fine), normalised where a weight is given and
        rotated to row_pos (int32 [n]).  Returns (q_out, k_out), of out_dtype (by
        default the inputs' type); an output may be its input.  stream: the
        current one, unless given; the caller orders a given one after what makes
        the arguments and before what uses the results, and may drop its tensors
        once the call returns."""
        return load_calls().norm_rope(self.address, q, k, row_pos, q_weight, k_weight, q_out, k_out, out_dtype, stream)
