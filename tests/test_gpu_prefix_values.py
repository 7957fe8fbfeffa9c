"""Shared-prefix decode at the edges of its number types: what is not finite
shows in the outputs."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_OK
from rope_helpers import prefix_workload

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0


def decode(w, gs, pl, q, cache=None, tab=None):
    if cache is None:
        cache, tab = device_cache(w)
    out, lse = cache.decode_prefix(q, tab, to_dev(w.seq_lens), w.seq_lens, gs, pl, w.n_qtok, w.scale, out=torch.empty(w.q.shape, device="cuda"))
    torch.cuda.synchronize()
    assert cache.check() == PA_OK
    return out, lse


@pytest.mark.parametrize("t", [1, 3])
@pytest.mark.parametrize("where", ["prefix", "suffix"])
def test_a_nan_key_shows_in_every_row_that_sees_it(where, t):
    """One NaN in a stored key of one head, in a batch that many CTAs split: every
    query row of that head that sees the key is NaN, and no other."""
    w, gs, pl = prefix_workload([(3, 2500), (2, 300)], [400, 30, 200, 50, 60], 16, F16, F16, n_qtok=t)
    q = to_dev(w.q).half()
    want, want_lse = decode(w, gs, pl, q)
    k = w.k_rows.copy()
    # rows are stored sequence after sequence, a sequence's prefix first
    row = 1300 if where == "prefix" else 2500 + 400 + 2500 + 7
    hit = [0, 1, 2] if where == "prefix" else [1]
    if where == "prefix":  # the copy that the first sequence's table row leads to, and the same in the others
        for a in (1300, 2900 + 1300, 2900 + 2530 + 1300):
            k[a, 2].view(np.uint16)[100] = 0x7e00
    else:
        k[row, 2].view(np.uint16)[100] = 0x7e00
    bad = W.Workload(w.name, w.seq_lens, t, w.page_size, w.n_blocks, F16, F16, w.table, k, w.v_rows, w.q, w.scale)
    out, lse = decode(bad, gs, pl, q)
    mark = torch.zeros(5, t, 24, dtype=torch.bool, device="cuda")
    mark[hit, :, 12:18] = True
    assert out[mark].isnan().all() and lse[mark].isnan().all()
    assert torch.equal(out[~mark], want[~mark]) and torch.equal(lse[~mark], want_lse[~mark])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_a_nan_query_row_is_nan(dtype):
    """And not a row that sees no key (zeros, lse -inf)."""
    w, gs, pl = prefix_workload([(3, 2500), (2, 300)], [400, 30, 200, 50, 60], 16, Q8, Q4)
    q = to_dev(w.q).to(dtype)
    want, want_lse = decode(w, gs, pl, q)
    q[1, 0, 7, 33] = float("nan")
    out, lse = decode(w, gs, pl, q)
    mark = torch.zeros(5, 1, 24, dtype=torch.bool, device="cuda")
    mark[1, 0, 7] = True
    assert out[mark].isnan().all() and lse[mark].isnan().all()
    assert torch.equal(out[~mark], want[~mark]) and torch.equal(lse[~mark], want_lse[~mark])
