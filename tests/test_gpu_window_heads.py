"""Windowed attention of pools with other numbers of KV heads than four: a rank's share of the heads, or more."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import assert_close, assert_lse_close, to_dev
from paged_kv_gqa_11_gb300 import PA_OK
from paged_kv_gqa_11_gb300.cache import PagedKVCache

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0


def attend64(q, k, v, lens, n_new, window, sinks):
    """(out, lse) by the definition in float64, from k and v [rows][heads][256]."""
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    at = row = 0
    for n, length in zip(n_new, lens):
        for i in range(n):
            p = int(length) - n + i
            x = np.arange(p + 1)
            x = row + x[(x > p - (window or p + 1)) | (x < sinks)]
            z = np.einsum("hgd,xhd->hgx", q[at + i].reshape(-1, 6, 256), k[x]) / 16.0
            m = z.max(-1, keepdims=True)
            e = np.exp(z - m)
            s = e.sum(-1, keepdims=True)
            out[at + i] = np.einsum("hgx,xhd->hgd", e / s, v[x]).reshape(-1, 256)
            lse[at + i] = (m + np.log(s)).reshape(-1)
        at += n
        row += int(length)
    return out, lse


@pytest.mark.parametrize("heads", [1, 2, 3, 8])
@pytest.mark.parametrize("kt,vt", [(F16, Q8), (Q8, Q4)])
@pytest.mark.parametrize("lens,n_new,window,sinks", [
    ([700, 40, 900], [1, 5, 33], 300, 4),
    ([700, 300, 64, 900], [150, 1, 64, 200], 100, 20),  # prompts whose windows begin on both sides of the sinks' end
    ([400], [400], 0, 0),
    ([300 + i % 5 for i in range(304)], [1] * 304, 64, 4),  # single tokens, one CTA or a cluster to a segment
    ([1500 + i % 5 for i in range(36)], [1] * 36, 0, 0),
])
def test_other_numbers_of_heads(heads, kt, vt, lens, n_new, window, sinks):
    rng = np.random.default_rng(heads)
    lens = np.array(lens if heads < 8 or len(lens) < 100 else lens[:70], np.int32)
    n_new = np.array(n_new[:len(lens)], np.int32)
    rows, tokens, page = int(lens.sum()), int(n_new.sum()), 16
    pages = [-(-int(n) // page) for n in lens]
    order = rng.permutation(sum(pages)).tolist()
    table = W.table_from_lists([[order.pop() for _ in range(n)] for n in pages])
    stored = [W.random_rows(rng, rows, t, hkv=heads) for t in (kt, vt)]
    q = rng.standard_normal((tokens, 6 * heads, 256), dtype=np.float32)
    cache = PagedKVCache(sum(pages), page, kt, vt, n_kv_heads=heads)
    dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731
    cache.append(to_dev(stored[0]), to_dev(stored[1]), dev(np.repeat(np.arange(len(lens)), lens)),
                 dev(np.concatenate([np.arange(n) for n in lens])), dev(table))
    out, lse = cache.attend_window(to_dev(q).half(), dev(table), dev(lens), lens, n_new, window, sinks)
    torch.cuda.synchronize()
    assert cache.check() == PA_OK
    k, v = (oracle.dequant_rows(x.reshape(rows * heads, -1), t).reshape(rows, heads, 256) for x, t in zip(stored, (kt, vt)))
    want, want_lse = attend64(q.astype(np.float16).astype(np.float64), k, v, lens, n_new, window, sinks)
    assert_close(out.float().cpu().numpy(), want)
    assert_lse_close(lse.cpu().numpy(), want_lse)
