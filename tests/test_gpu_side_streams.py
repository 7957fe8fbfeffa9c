"""Calls on a stream that is passed in: what they read stays until they have read
it, what they return until the current stream has."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_OK
from paged_kv_gqa_11_gb300.cache import PagedKVCache
from paged_kv_gqa_11_gb300.rope import Rope
from rope_helpers import inv_freq, prefix_workload

pytestmark = pytest.mark.gpu
Q8 = W.TYPE_Q8_0


def busy(side):
    """Some 50 ms of work on `side`, after what the current stream has so far."""
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)


def overwrite(n):
    """Blocks that the allocator hands out next on the current stream, filled with ones."""
    keep = [torch.ones(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.current_stream().synchronize()
    return keep


def test_inputs_freed_before_the_kernel_runs():
    """Inputs made for the call and dropped with it, while the stream passed in is busy:
    their memory is not handed out again before the kernel has read it."""
    rng = np.random.default_rng(4)
    x0 = torch.from_numpy(rng.standard_normal((4096, 32, 256)).astype(np.float32)).cuda().half()
    pos, w = torch.arange(4096, dtype=torch.int32, device="cuda"), torch.rand(256, device="cuda").half()
    r, side = Rope(inv_freq(64)), torch.cuda.Stream()
    want, _ = r.apply(x0, None, pos, w)
    n = x0.numel() * 2
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = x0.clone()
    busy(side)
    got, _ = r.apply(x, None, pos, w, stream=side)
    del x
    keep = overwrite(n)
    side.synchronize()
    assert torch.equal(got, want)
    del keep
    # the append's queries and rows, and what it appends
    seq = torch.zeros(4096, dtype=torch.int32, device="cuda")
    tab = torch.arange(256, dtype=torch.int32, device="cuda")[None]
    a, b = PagedKVCache(256, 16, Q8, Q8), PagedKVCache(256, 16, Q8, Q8)
    want = a.append_rope(r, x0[:, 24:28], x0[:, 28:], seq, pos, tab, q=x0[:, :24])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = x0.clone()
    busy(side)
    got = b.append_rope(r, x[:, 24:28], x[:, 28:], seq, pos, tab, q=x[:, :24], stream=side)
    del x
    keep = overwrite(n)
    side.synchronize()
    assert a.check() == PA_OK and b.check() == PA_OK
    assert torch.equal(got, want) and torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)


def test_queries_of_a_shared_prefix_decode_freed_before_it_runs():
    w, gs, pl = prefix_workload([(40, 100)], [30] * 40, 16, Q8, Q8)
    cache, tab = device_cache(w)
    q0, sl, side = to_dev(w.q).half(), to_dev(w.seq_lens), torch.cuda.Stream()
    want, want_lse = cache.decode_prefix(q0, tab, sl, w.seq_lens, gs, pl, 1, w.scale)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    q = q0.clone()
    busy(side)
    out, lse = cache.decode_prefix(q, tab, sl, w.seq_lens, gs, pl, 1, w.scale, stream=side)
    del q
    keep = overwrite(q0.numel() * 2)
    side.synchronize()
    del keep
    assert cache.check() == PA_OK
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_results_dropped_before_the_current_stream_has_read_them():
    rng = np.random.default_rng(5)
    xs = [torch.from_numpy(rng.standard_normal((2048, 32, 256)).astype(np.float32)).cuda().half() for _ in range(2)]
    pos = torch.arange(2048, dtype=torch.int32, device="cuda")
    r, side, now = Rope(inv_freq(64)), torch.cuda.Stream(), torch.cuda.current_stream()
    want = r.apply(xs[0], None, pos)[0].clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got, _ = r.apply(xs[0], None, pos, stream=side)
    now.wait_stream(side)
    torch.cuda._sleep(100_000_000)
    copy = got.clone()
    del got
    later, _ = r.apply(xs[1], None, pos, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and not torch.equal(later, want)


def test_a_stream_passed_in_while_capturing():
    """A branch of a captured graph: forked from the capturing stream, joined to it, the
    call's inputs and results dropped inside."""
    rng = np.random.default_rng(6)
    xs = [torch.from_numpy(rng.standard_normal((64, 32, 256)).astype(np.float32)).cuda().half() for _ in range(2)]
    pos, w = torch.arange(64, dtype=torch.int32, device="cuda"), torch.rand(256, device="cuda").half()
    r, side = Rope(inv_freq(64)), torch.cuda.Stream()
    want = [r.apply(x * 2, None, pos, w)[0] + 1 for x in xs]
    x = xs[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        now = torch.cuda.current_stream()
        twice = x * 2
        side.wait_stream(now)
        y, _ = r.apply(twice, None, pos, w, stream=side)
        del twice
        scratch = torch.zeros_like(x)  # would take the dropped block
        now.wait_stream(side)
        out = y + 1
        del y, scratch
    for src, ref in zip(xs, want):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
