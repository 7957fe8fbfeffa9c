"""Windowed attention over caches that hold infinite values: which tokens they reach."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_OK
from window_helpers import window_batch

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0


def infinite(t):
    """A stored row of 256 values past binary16's range."""
    if t == F16:
        return np.tile(np.array([0x00, 0x7c], np.uint8), 256)
    scale = np.array([600.0 if t == Q8 else 60000.0], np.float16).view(np.uint8)  # times 127, times 7
    return np.tile(np.concatenate([scale, np.full(32 if t == Q8 else 16, 127 if t == Q8 else 255, np.uint8)]), 8)


def reached(n_new, lens, window, sinks, bad):
    """Of every token whether it sees one of its sequence's bad keys, and how far the nearest bad one is that it does not."""
    sees, far = [], []
    for n, length, keys in zip(n_new, lens, bad):
        for p in range(length - n, length):
            lo = max(0, p - window + 1) if window else 0
            sees.append(any(k <= p and (k >= lo or k < sinks) for k in keys))
            far.append(min([k - p if k > p else lo - k for k in keys if k > p or sinks <= k < lo], default=1 << 30))
    return np.array(sees), np.array(far)


def check(kt, vt, lens, n_new, window, sinks, bad, reach):
    """Tokens that see a bad value have it in their results; those farther than `reach` from one have the bits that they have
    without it; nobody's lse knows of it."""
    w = window_batch(lens, n_new, 16, kt, vt, seed=window + sinks)
    rows = w.v_rows.copy()
    for start, keys in zip(np.cumsum([0, *lens]), bad):
        for k in keys:
            rows[start + k] = infinite(vt)
    res = []
    for v in (w.v_rows, rows):
        cache, tab = device_cache(W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, kt, vt, w.table, w.k_rows, v, w.q, w.scale))
        res.append(cache.attend_window(to_dev(w.q), tab, to_dev(w.seq_lens), w.seq_lens, np.asarray(n_new, np.int32), window, sinks, w.scale))
        torch.cuda.synchronize()
        assert cache.check() == PA_OK
    (plain, plain_lse), (out, lse) = res
    assert torch.equal(lse, plain_lse)
    sees, far = reached(n_new, lens, window, sinks, bad)
    clean = to_dev(~sees & (far > reach))
    assert clean.any() and not torch.isfinite(out[to_dev(sees)]).any()
    assert torch.isfinite(out[clean]).all() and torch.equal(out[clean], plain[clean])


@pytest.mark.parametrize("kt,vt", [(F16, F16), (Q8, Q8), (Q8, Q4)])
@pytest.mark.parametrize("lens,n_new,window,sinks,bad", [
    ([1500], [1500], 256, 4, [[4]]),  # the first tokens see it, behind the sinks, the later ones do not
    ([1000], [1000], 40, 1, [[1, 15, 16, 500, 999]]),
    ([900, 40], [700, 40], 100, 17, [[17, 31, 450], []]),  # no new token sees the first two
    ([700], [690], 16, 20, [[20, 31]]),
    ([600], [600], 30, 0, [[0, 300]]),
    ([1300, 640, 700], [1290, 64, 700], 300, 129, [[130, 143, 400], [143], [143]]),
    ([500], [500], 16, 15, [[15]]),
])
def test_prompts(kt, vt, lens, n_new, window, sinks, bad):
    check(kt, vt, lens, n_new, window, sinks, bad, 64)


@pytest.mark.parametrize("kt,vt", [(F16, F16), (Q8, Q4), (Q4, Q8)])
@pytest.mark.parametrize("lens,n_new,window,sinks,bad", [
    ([400, 63, 300], [63, 63, 2], 20, 4, [[4, 15, 350], [4, 30], [4, 200]]),
    ([63], [63], 8, 1, [[1, 15, 40]]),
])
def test_few_tokens(kt, vt, lens, n_new, window, sinks, bad):
    check(kt, vt, lens, n_new, window, sinks, bad, 11)  # the tokens of 64 query rows lie up to 11 apart


@pytest.mark.parametrize("vt", [Q8, Q4])
def test_single_tokens(vt):
    lens = [600 + i % 9 for i in range(64)]
    check(Q8, vt, lens, [1] * 64, 400, 5, [[n - 1 - 400 * (i % 2), 5, 15, 100] if i % 3 else [5] for i, n in enumerate(lens)], 0)
