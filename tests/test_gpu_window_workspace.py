"""Windowed attention in scratch that the caller sized once, and as a process's first call of the library inside a capture."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import workloads as W
from conftest import ROOT
from gpu_helpers import device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_OK, pa_attend_window_workspace_size
from window_helpers import window_batch

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0


@pytest.mark.parametrize("kt,vt", [(F16, F16), (Q8, Q4)])
@pytest.mark.parametrize("window,sinks", [(100, 0), (64, 5), (0, 0), (300, 33)])
def test_one_scratch_for_every_smaller_batch(kt, vt, window, sinks):
    """Sized for the largest batch, used by smaller ones; what lies behind it stays."""
    most = np.array([200, 70, 63], np.int32)
    longest = np.array([700, 400, 300], np.int32)
    w0 = window_batch(longest, most, 16, kt, vt)
    size = pa_attend_window_workspace_size(device_cache(w0)[0].pool, longest, most, window, sinks)
    room = torch.full((size + 4096,), 171, dtype=torch.uint8, device="cuda")
    for n_new, less in (([200, 70, 63], 0), ([200, 70, 63], 1), ([200, 64, 63], 7), ([64, 63, 63], 12), ([100, 63, 1], 15), ([63, 63, 0], 3),
                        ([199, 69, 5], 25), ([1, 1, 1], 100)):
        w = window_batch(longest - less, n_new, 16, kt, vt, seed=less)
        cache, tab = device_cache(w)
        call = lambda **kw: cache.attend_window(to_dev(w.q).half(), tab, to_dev(w.seq_lens), w.seq_lens,  # noqa: E731
                                                np.array(n_new, np.int32), window, sinks, **kw)
        want, want_lse = call()
        out, lse = call(workspace=room[:size])
        torch.cuda.synchronize()
        assert cache.check() == PA_OK and torch.equal(out, want) and torch.equal(lse, want_lse)
        assert (room[size:] == 171).all()


FIRST = """
import numpy as np, torch
from paged_kv_gqa_11_gb300.cache import PagedKVCache
lens, n_new = np.array({lens}, np.int32), np.array({n_new}, np.int32)
n = len(lens)
cache = PagedKVCache(n * 8, 64, 8, 2)
cache.k_pool.random_(0, 60), cache.v_pool.random_(0, 60)
table = torch.arange(n * 8, dtype=torch.int32, device="cuda").reshape(n, 8)
q = torch.randn(int(n_new.sum()), 24, 256, device="cuda").half()
dev = torch.from_numpy(lens).cuda()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = cache.attend_window(q, table, dev, lens, n_new, 200, 4)
g.replay()
torch.cuda.synchronize()
want, want_lse = cache.attend_window(q, table, dev, lens, n_new, 200, 4)
assert cache.check() == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
print("done")
"""


@pytest.mark.parametrize("lens,n_new", [([500] * 64, [1] * 64), ([500, 300, 200], [100, 5, 1])])
def test_first_call_of_a_process_inside_a_capture(lens, n_new):
    r = subprocess.run([sys.executable, "-c", FIRST.format(lens=lens, n_new=n_new)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]
