"""Decode with shared prefixes against the float64 oracle, which knows nothing
of the sharing (each sequence's own table over all its rows)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import assert_close, assert_lse_close, device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_ERR_BOUNDS, PA_OK, PaError, pa_decode_prefix_workspace_size
from paged_kv_gqa_11_gb300.cache import PagedKVCache
from paged_kv_gqa_11_gb300.rope import Rope
from rope_helpers import inv_freq, prefix_workload

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0
THREADS = 8


def run(w, gs, pl, dtype=torch.float32, cache=None, tab=None, **kw):
    if cache is None:
        cache, tab = device_cache(w)
    q = to_dev(w.q).to(dtype)
    out, lse = cache.decode_prefix(q, tab, to_dev(w.seq_lens), w.seq_lens, gs, pl, w.n_qtok, w.scale, **kw)
    torch.cuda.synchronize()
    assert cache.check() == PA_OK
    return out, lse, q


def against_oracle(w, gs, pl, dtype=torch.float32, what=""):
    out, lse, q = run(w, gs, pl, dtype)
    ref = W.Workload(w.name, w.seq_lens, w.n_qtok, w.page_size, w.n_blocks, w.k_type, w.v_type, w.table, w.k_rows, w.v_rows,
                     q.float().cpu().numpy(), w.scale)
    want, want_lse = oracle.decode_workload(ref, n_threads=THREADS)
    assert_close(out.float().cpu().numpy(), want, what=what)
    assert_lse_close(lse.cpu().numpy(), want_lse, what=what)


@pytest.mark.parametrize("kt", [F16, Q4, Q8])
@pytest.mark.parametrize("vt", [F16, Q4, Q8])
def test_every_format_pair(kt, vt):
    w, gs, pl = prefix_workload([(3, 200)], [50, 1, 130], 16, kt, vt)
    against_oracle(w, gs, pl, torch.float16)


@pytest.mark.parametrize("p", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400])
def test_prefix_lengths(p):
    """Prefixes that end before, at and after every tile and page edge; suffixes of one row and more."""
    w, gs, pl = prefix_workload([(2, p), (3, p + 3)], [1, 17, 129, 64, 2], 48, Q8, Q4, seed=p)
    against_oracle(w, gs, pl, torch.bfloat16, what=f"prefix {p}")


@pytest.mark.parametrize("t", [1, 2, 3, 5, 8, 11, 20, 96])
def test_query_tokens(t):
    """Causal among the new tokens; a sequence whose own rows are the new tokens alone."""
    w, gs, pl = prefix_workload([(3, 333), (1, 40)], [t, t + 1, t + 140, t + 9], 16, Q8, Q8, n_qtok=t, seed=t)
    against_oracle(w, gs, pl, what=f"{t} tokens")


@pytest.mark.parametrize("b,t", [(10, 1), (11, 1), (17, 1), (22, 1), (40, 1), (9, 4), (2, 33)])
def test_many_query_rows(b, t):
    """Groups of more query rows than one row tile holds."""
    w, gs, pl = prefix_workload([(b, 290)], [t + (7 * i) % 40 for i in range(b)], 32, Q4, Q4, n_qtok=t, seed=b)
    against_oracle(w, gs, pl, torch.float16, what=f"{b} x {t}")


@pytest.mark.parametrize("qt,ot", [("float32", "float16"), ("float16", "float32"), ("bfloat16", "float16")])
def test_types_of_queries_and_outputs(qt, ot):
    w, gs, pl = prefix_workload([(4, 150)], [20, 30, 40, 50], 64, Q8, Q8, n_qtok=2)
    cache, tab = device_cache(w)
    out = torch.full(w.q.shape, float("nan"), dtype=getattr(torch, ot), device="cuda")
    got, lse, q = run(w, gs, pl, getattr(torch, qt), cache, tab, out=out)
    assert got is out
    same, lse2, _ = run(w, gs, pl, getattr(torch, qt), cache, tab)
    assert torch.equal(lse, lse2)
    f32 = torch.empty(w.q.shape, device="cuda")
    run(w, gs, pl, getattr(torch, qt), cache, tab, out=f32)
    assert torch.equal(f32.to(out.dtype), out) and torch.equal(f32.to(same.dtype), same)


def test_mixed_groups_and_long_prefix():
    """A long prefix that many CTAs split, singles, groups without a prefix, in one batch."""
    w, gs, pl = prefix_workload([(1, 700), (8, 9000), (2, 0), (4, 513), (1, 0)], [300, 5, 900, 1, 64, 65, 2000, 16, 3, 70, 1, 40, 128, 10, 20, 600],
                                16, Q4, Q4)
    against_oracle(w, gs, pl, torch.float16)


def test_the_benchmark_batch():
    w = W.shared_prefix(n_seq=8, prefix=4096, own=300)
    gs, pl = np.array([8], np.uint32), np.array([4096], np.int32)
    against_oracle(w, gs, pl)


def test_more_sequences_than_a_launch_takes():
    """300 sequences, a group across the cut between sub-batches."""
    own = [3 + (11 * i) % 60 for i in range(300)]
    w, gs, pl = prefix_workload([(2, 40), (251, 70), (47, 100)], own, 16, Q8, Q4)
    against_oracle(w, gs, pl, torch.float16)


@pytest.mark.parametrize("kind", ["rising", "late", "scales"])
@pytest.mark.parametrize("t", [1, 4])
def test_stress_inputs(kind, t):
    """Logits that grow along the sequence, pieces whose maxima lie far apart,
    zero and subnormal scales: one sequence, its first 1504 rows as the prefix of two
    copies."""
    base = W.stress_workload(kind, 77, [3000], 16, Q8, Q4, t)
    rows = 1504
    n = 3000
    pages = -(-n // 16)
    table = np.stack([np.arange(pages), np.concatenate([np.arange(rows // 16), pages + np.arange(pages - rows // 16)])]).astype(np.int32)
    w = W.Workload(kind, np.array([n, n], np.int32), t, 16, 2 * pages, Q8, Q4, table, np.concatenate([base.k_rows] * 2),
                   np.concatenate([base.v_rows] * 2), np.concatenate([base.q, base.q]), base.scale)
    against_oracle(w, np.array([2], np.uint32), np.array([rows], np.int32), what=kind)


@pytest.mark.parametrize("kt,vt,t,ps,groups", [
    (Q4, Q4, 1, 16, [(14, 1500), (2, 1000), (5, 130), (1, 300), (12, 2100), (6, 0)]),
    (Q8, Q4, 2, 48, [(9, 1500), (2, 1000), (5, 130), (1, 300), (7, 2100), (6, 0)]),
    (F16, F16, 1, 64, [(8, 2500), (3, 1000), (6, 1200)]),
    (Q8, Q8, 11, 16, [(3, 900), (1, 20), (4, 400)]),
    (Q4, Q8, 1, 16, [(30, 128)] + [(2, 16 + 16 * i) for i in range(25)]),
])
def test_ctas_of_many_pieces(kt, vt, t, ps, groups):
    """Several tiles and pieces to a CTA: wide and narrow ones in turn, pieces
    of one tile, and all numbers of threads that the merge gives a row."""
    own = [t + (97 * i) % 800 for i in range(sum(b for b, _ in groups))]
    w, gs, pl = prefix_workload(groups, own, ps, kt, vt, n_qtok=t, seed=t)
    against_oracle(w, gs, pl, torch.float16)


@pytest.mark.parametrize("kind", ["rising", "late", "scales"])
@pytest.mark.parametrize("t", [1, 4])
def test_references_raised_inside_a_piece(kind, t):
    """The stress inputs again, long enough that a CTA's piece has several tiles:
    weights already in O are scaled down, tiles whose weights overflow are redone."""
    base = W.stress_workload(kind, 78, [12000], 16, Q8, Q4, t)
    n, rows, pages = 12000, 6000, 750
    table = np.stack([np.arange(pages), np.concatenate([np.arange(rows // 16), pages + np.arange(pages - rows // 16)])]).astype(np.int32)
    w = W.Workload(kind, np.array([n, n], np.int32), t, 16, 2 * pages, Q8, Q4, table, np.concatenate([base.k_rows] * 2),
                   np.concatenate([base.v_rows] * 2), np.concatenate([base.q, base.q]), base.scale)
    against_oracle(w, np.array([2], np.uint32), np.array([rows], np.int32), what=kind)


def test_page_size_and_placement_change_nothing():
    outs = []
    for ps in (16, 48, 256):
        w, gs, pl = prefix_workload([(3, 515)], [200, 31, 77], ps, Q8, Q8, seed=9)
        outs.append(run(w, gs, pl)[:2])
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("kt,vt", [(F16, F16), (Q8, Q4), (Q4, Q8)])
def test_rows_past_the_ends_do_not_count(kt, vt):
    """Every byte of the pools that no live row owns is NaN (0x7f7f scales and
    halves are huge or NaN): nothing of it reaches an output."""
    w, gs, pl = prefix_workload([(2, 133), (1, 9)], [5, 40, 30], 64, kt, vt)
    want, want_lse, _ = run(w, gs, pl)
    c = PagedKVCache(w.n_blocks, w.page_size, kt, vt)
    c.k_pool.fill_(0x7f), c.v_pool.fill_(0x7f)
    tab = to_dev(w.table)
    c.append(to_dev(w.k_rows), to_dev(w.v_rows), to_dev(w.row_seq), to_dev(w.row_pos), tab)
    out, lse, _ = run(w, gs, pl, cache=c, tab=tab)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_bad_table_entries_are_reported():
    """Entries outside the pool, in a prefix and in a suffix: finite outputs, the
    report, and sequences of other groups untouched."""
    w, gs, pl = prefix_workload([(2, 100), (2, 64)], [40, 50, 30, 20], 16, Q8, Q4)
    good, good_lse, _ = run(w, gs, pl)
    cache, _ = device_cache(w)
    for s, e, v in ((0, 2, w.n_blocks), (1, 7, -5), (1, 8, 2 ** 31 - 1)):
        t = w.table.copy()
        t[s, e] = v
        out, lse = cache.decode_prefix(to_dev(w.q), to_dev(t), to_dev(w.seq_lens), w.seq_lens, gs, pl, 1, w.scale)
        torch.cuda.synchronize()
        assert cache.check() == PA_ERR_BOUNDS
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        assert torch.equal(out[2:], good[2:]) and torch.equal(lse[2:], good_lse[2:])


def test_device_lengths_are_checked():
    w, gs, pl = prefix_workload([(3, 100)], [40, 50, 30], 16, Q8, Q4)
    good, good_lse, _ = run(w, gs, pl)
    cache, tab = device_cache(w)
    dev = w.seq_lens.copy()
    dev[1] += 1
    out, lse = cache.decode_prefix(to_dev(w.q), tab, to_dev(dev), w.seq_lens, gs, pl, 1, w.scale)
    torch.cuda.synchronize()
    assert cache.check() == PA_ERR_BOUNDS
    assert not out[1].any() and (lse[1] == float("-inf")).all()
    for i in (0, 2):
        assert torch.equal(out[i], good[i]) and torch.equal(lse[i], good_lse[i])


@pytest.mark.parametrize("t", [1, 3, 20])
def test_nothing_is_written_past_the_buffers(t):
    w, gs, pl = prefix_workload([(5, 200), (1, 10)], [t, t + 5, t + 100, t + 3, t + 1, t + 7], 16, Q8, Q8, n_qtok=t)
    cache, tab = device_cache(w)
    want, want_lse, q = run(w, gs, pl, torch.float16, cache, tab)
    need = pa_decode_prefix_workspace_size(cache.pool, w.n_seq, len(gs), t)
    n, m = want.numel(), want_lse.numel()
    out = torch.full((n + 4096,), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((m + 1024,), 7.0, device="cuda")
    ws = torch.full((need + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    pools = cache.k_pool.clone(), cache.v_pool.clone()
    cache.decode_prefix(q, tab, to_dev(w.seq_lens), w.seq_lens, gs, pl, t, w.scale, out=out[:n].view(want.shape),
                        lse=lse[:m].view(want_lse.shape), workspace=ws[:need])
    torch.cuda.synchronize()
    assert cache.check() == PA_OK
    assert torch.equal(out[:n].view(want.shape), want) and torch.equal(lse[:m].view(want_lse.shape), want_lse)
    assert (out[n:] == 7).all() and (lse[m:] == 7).all() and (ws[need:] == 0x5a).all()
    assert torch.equal(pools[0], cache.k_pool) and torch.equal(pools[1], cache.v_pool)
    # a workspace one byte short is refused
    with pytest.raises(PaError):
        cache.decode_prefix(q, tab, to_dev(w.seq_lens), w.seq_lens, gs, pl, t, w.scale, workspace=ws[:need - 1])


def test_captured_twice_and_on_two_streams():
    """Two captured graphs of one cache replayed at the same time on two streams,
    and calls on a side stream, equal the plain call."""
    w, gs, pl = prefix_workload([(6, 3000)], [100, 200, 30, 40, 50, 1000], 16, Q4, Q4)
    cache, tab = device_cache(w)
    sl = to_dev(w.seq_lens)
    q = [to_dev(w.q).half() * f for f in (1.0, 0.5)]
    want = [cache.decode_prefix(x, tab, sl, w.seq_lens, gs, pl, 1, w.scale) for x in q]
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(cache.decode_prefix(x, tab, sl, w.seq_lens, gs, pl, 1, w.scale))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    res = [cache.decode_prefix(x, tab, sl, w.seq_lens, gs, pl, 1, w.scale, stream=s) for x, s in zip(q, streams)]
    torch.cuda.synchronize()
    for a, b in zip(res, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert cache.check() == PA_OK


def test_a_serving_step_from_projections():
    """Eight continuations of one prompt, step by step as a server runs them, no
    synchronisation in between: the projection's rows appended (normalised and
    rotated, the queries with them), then the shared-prefix decode.  Every step
    equals pa_decode and, at the end, the oracle on the rows the cache holds."""
    rng = np.random.default_rng(12)
    n, prefix, steps, ps = 8, 200, 5, 16
    r = Rope(inv_freq(64))
    wq, wk = (torch.from_numpy((1 + 0.2 * rng.standard_normal(256)).astype(np.float32)).cuda().half() for _ in range(2))
    pages, shared = 16, prefix // ps
    table = np.zeros((n, pages), np.int32)
    table[:, :shared] = np.arange(shared)
    table[:, shared:] = shared + np.arange(n * (pages - shared)).reshape(n, -1)
    c = PagedKVCache(shared + n * (pages - shared), ps, Q8, Q8)
    tab = to_dev(table)
    proj = torch.from_numpy(rng.standard_normal((prefix, 32, 256)).astype(np.float32)).cuda().half()
    # the prompt: into the shared pages once, its tail into every sequence's own page
    for s in range(n):
        a = 0 if s == 0 else shared * ps
        m = prefix - a
        c.append_rope(r, proj[a:, 24:28], proj[a:, 28:], torch.full((m,), s, dtype=torch.int32, device="cuda"),
                      torch.arange(a, prefix, dtype=torch.int32, device="cuda"), tab, k_weight=wk)
    seq = torch.arange(n, dtype=torch.int32, device="cuda")
    gs, pl = np.array([n], np.uint32), np.array([prefix], np.int32)
    results = []
    for i in range(steps):
        x = torch.from_numpy(rng.standard_normal((n, 32, 256)).astype(np.float32)).cuda().half()
        lens = np.full(n, prefix + i + 1, np.int32)
        q = c.append_rope(r, x[:, 24:28], x[:, 28:], seq, torch.full_like(seq, prefix + i), tab, k_weight=wk, q=x[:, :24], q_weight=wq)
        out, lse = c.decode_prefix(q[:, None], tab, to_dev(lens), lens, gs, pl, 1)
        ref, ref_lse = c.decode(q[:, None].float(), tab, to_dev(lens), lens, 1)
        results.append((out, lse, ref, ref_lse))
    torch.cuda.synchronize()
    assert c.check() == PA_OK
    for out, lse, ref, ref_lse in results:
        assert_close(out.float().cpu().numpy(), ref.double().cpu().numpy())
        assert_lse_close(lse.cpu().numpy(), ref_lse.double().cpu().numpy())
    k, v = c.read_rows(torch.repeat_interleave(seq, prefix + steps), torch.arange(prefix + steps, dtype=torch.int32, device="cuda").repeat(n), tab,
                       dtype=torch.float32)
    k, v = (y.double().cpu().numpy().reshape(n, prefix + steps, 4, 256) for y in (k, v))
    z = np.einsum("nhgd,nlhd->nhgl", q.double().cpu().numpy().reshape(n, 4, 6, 256), k) / 16
    e = np.exp(z - z.max(-1, keepdims=True))
    want = np.einsum("nhgl,nlhd->nhgd", e / e.sum(-1, keepdims=True), v).reshape(n, 1, 24, 256)
    assert_close(out.float().cpu().numpy(), want)


def test_refusals_of_the_python_call():
    """Arguments of the wrong type, shape, place or device: PaError, nothing written, and the next call works."""
    w, gs, pl = prefix_workload([(2, 100), (1, 3)], [40, 50, 30], 16, Q8, Q4)
    cache, tab = device_cache(w)
    q, sl = to_dev(w.q).half(), to_dev(w.seq_lens)
    want, want_lse = cache.decode_prefix(q, tab, sl, w.seq_lens, gs, pl, 1, w.scale)
    out = torch.full_like(q, 7.0)
    good = dict(q=q, block_table=tab, seq_lens_dev=sl, seq_lens_host=w.seq_lens, group_sizes=gs, prefix_lens=pl, n_qtok=1, scale=w.scale, out=out)
    bad = [
        dict(q=q.double()), dict(q=q[:, :, ::2]), dict(q=q.cpu()), dict(q=q[0]), dict(q=q[..., :128].contiguous()), dict(q=None), dict(q=w.q),
        dict(block_table=tab.long()), dict(block_table=tab.T), dict(block_table=tab[:2]), dict(block_table=tab.cpu()), dict(block_table=tab[:, :1].contiguous()),
        dict(seq_lens_dev=sl.long()), dict(seq_lens_dev=sl[:2]), dict(seq_lens_dev=w.seq_lens),
        dict(seq_lens_host=w.seq_lens.astype(np.int64)), dict(seq_lens_host=w.seq_lens[:2]), dict(seq_lens_host=sl), dict(seq_lens_host=w.seq_lens * 0),
        dict(seq_lens_host=np.repeat(w.seq_lens, 2)[::2]), dict(seq_lens_host=w.seq_lens.astype(np.float32)),
        dict(group_sizes=gs + 1), dict(group_sizes=gs[:1]), dict(group_sizes=np.array([3, 0], np.uint32)), dict(prefix_lens=pl + 1000),
        dict(prefix_lens=pl - 200), dict(prefix_lens=pl[:1]), dict(n_qtok=2), dict(n_qtok="1"), dict(scale="x"), dict(scale=0.0), dict(scale=float("nan")),
        dict(scale=float("inf")), dict(scale=-1.0), dict(out=out[:2]), dict(out=out.double()), dict(out=out.cpu()), dict(out=torch.empty(3, 1, 24, 512, device="cuda")[..., ::2]),
        dict(lse=torch.empty(3, 1, 24, device="cuda").half()), dict(lse=torch.empty(3, 24, device="cuda")), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        dict(workspace=torch.empty(1 << 24, dtype=torch.uint8)), dict(stream="s"), dict(stream=object()),
    ]
    for change in bad:
        with pytest.raises(PaError):
            cache.decode_prefix(**{**good, **change})
    torch.cuda.synchronize()
    assert (out == 7).all() and cache.check() == PA_OK
    got, lse = cache.decode_prefix(**good)
    assert got is out and torch.equal(out, want) and torch.equal(lse, want_lse)
