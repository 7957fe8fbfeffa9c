"""The norm and rotation in float64, and batches of sequences that share prefixes."""
from __future__ import annotations

import numpy as np

import workloads as W

THETA = 1e6


def inv_freq(rot: int, theta: float = THETA) -> list[float]:
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def norm_rope64(x, pos, freq, interleaved=False, w=None, eps=1e-6, offset=0.0, factor=1.0):
    """float64 heads [n][h][256] -> (result, |a| + |b| of the pair behind each value)."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * (np.asarray(w, np.float64) + offset)
    half, rot = len(freq), 2 * len(freq)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    c, s = factor * np.cos(ang), factor * np.sin(ang)
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(half), np.arange(half, rot))
    y, mag = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def prefix_workload(groups, own, ps, k_type, v_type, n_qtok=1, seed=5):
    """groups: [(sequences, prefix rows)]; own: rows that each sequence adds.  A
    prefix's whole pages are shared blocks, the page it ends in is every
    sequence's own copy; blocks are shuffled.  Returns (workload, group sizes,
    prefix lengths)."""
    rng = np.random.default_rng(seed)
    lens, k_rows, v_rows, lists, nxt, i = [], [], [], [], 0, 0
    for b, p in groups:
        pk, pv = W.random_rows(rng, p, k_type), W.random_rows(rng, p, v_type)
        whole = p // ps
        shared = list(range(nxt, nxt + whole))
        nxt += whole
        for _ in range(b):
            n = own[i]
            k_rows += [pk, W.random_rows(rng, n, k_type)]
            v_rows += [pv, W.random_rows(rng, n, v_type)]
            mine = -(-(p + n) // ps) - whole
            lists.append(shared + list(range(nxt, nxt + mine)))
            nxt += mine
            lens.append(p + n)
            i += 1
    # the queries before the placement, so that they do not depend on the page size
    q = rng.standard_normal((len(lens), n_qtok, W.HQ, W.D), dtype=np.float32)
    order = rng.permutation(nxt).tolist()
    table = W.table_from_lists([[order[x] for x in l] for l in lists])
    w = W.Workload("prefix", np.array(lens, np.int32), n_qtok, ps, nxt, k_type, v_type, table, np.concatenate(k_rows),
                   np.concatenate(v_rows), q)
    return w, np.array([b for b, _ in groups], np.uint32), np.array([p for _, p in groups], np.int32)
