"""Turned rows have the same bytes however a move is cut into calls: a row's key depends on its own
places alone, not on the rows beside it or the kernel that their number selects."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_OK
from paged_kv_gqa_11_gb300.rope import Rope
from window_helpers import window_batch

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0


@pytest.mark.parametrize("kt", [F16, Q8, Q4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_turned_rows_in_one_call_and_in_parts(kt, interleaved):
    """8000 rows down by 8777 places, in order, mixed with rows of other distances, in parts and few at a time; a last unit of a
    phase (2^-32 of a turn) changes about 10 of their 8 million binary16 keys."""
    n, by = 8000, 8777
    w = window_batch([by + n], [1], 16, kt, Q8, seed=11)
    rope = Rope.from_theta(256, 1e4, interleaved=interleaved)
    dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731

    def moved(parts, **kw):
        cache, tab = device_cache(w)
        for at in parts:
            zero = dev(np.zeros(len(at)))
            cache.move_rows(zero, dev(at + by), zero, dev(at), tab, rope=rope, **kw)
        torch.cuda.synchronize()
        assert cache.check() == PA_OK
        return cache

    at = np.arange(n)
    want = moved([at], disjoint=True)
    for parts, kw in (([at], {}), ([at[::-1].copy()], {"disjoint": True}), ([np.random.default_rng(1).permutation(n)], {}),
                      (np.split(at, [3, 1001, 1002, 5000]), {}), (np.array_split(at, 200), {})):
        got = moved(parts, **kw)
        assert torch.equal(got.k_pool, want.k_pool) and torch.equal(got.v_pool, want.v_pool)
