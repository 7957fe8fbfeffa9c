"""Ragged batches for the windowed attention, and the attention in float64."""
from __future__ import annotations

import numpy as np

import oracle
import workloads as W


def window_batch(lens, n_new, ps, k_type, v_type, seed=3):
    """A workload whose queries are rows, one sequence's new tokens after the other's: [tokens][24][256]."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    total = int(lens.sum())
    q = rng.standard_normal((int(np.sum(n_new)), W.HQ, W.D), dtype=np.float32)
    pages = [-(-int(n) // ps) for n in lens]
    order = rng.permutation(max(1, sum(pages))).tolist()
    lists, at = [], 0
    for n in pages:
        lists.append(order[at: at + n])
        at += n
    table = W.table_from_lists(lists, max(1, max(pages)))
    return W.Workload("window", lens, 1, ps, max(1, sum(pages)), k_type, v_type, table, W.random_rows(rng, total, k_type),
                      W.random_rows(rng, total, v_type), q)


def attend64(w, n_new, window, sinks, q=None, k=None, v=None):
    """(out [tokens][24][256], lse [tokens][24]) by the definition, from the stored rows (or k, v [rows][4][256])."""
    q = np.asarray(w.q if q is None else q, np.float64)
    rows = lambda x, t: oracle.dequant_rows(x.reshape(-1, x.shape[-1]), t).reshape(len(x), W.HKV, W.D)  # noqa: E731
    k = rows(w.k_rows, w.k_type) if k is None else np.asarray(k, np.float64)
    v = rows(w.v_rows, w.v_type) if v is None else np.asarray(v, np.float64)
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    at = row = 0
    for n, length in zip(n_new, w.seq_lens):
        for i in range(n):
            p = int(length) - n + i
            x = np.arange(p + 1)
            if window:
                x = x[(x > p - window) | (x < sinks)]
            ks, vs = k[row + x], v[row + x]
            for h in range(W.HKV):
                z = q[at + i, 6 * h: 6 * h + 6] @ ks[:, h].T * w.scale
                m = z.max(-1, keepdims=True)
                e = np.exp(z - m)
                s = e.sum(-1, keepdims=True)
                out[at + i, 6 * h: 6 * h + 6] = e @ vs[:, h] / s
                lse[at + i, 6 * h: 6 * h + 6] = (m + np.log(s))[:, 0]
        at += n
        row += int(length)
    return out, lse
