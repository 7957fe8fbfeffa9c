"""Rows and blocks moved within the cache: bytes where nothing is turned, and turned keys
against float64."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_ERR_BOUNDS, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_OK, PaError
from paged_kv_gqa_11_gb300.cache import PagedKVCache
from paged_kv_gqa_11_gb300.rope import Rope
from rope_helpers import inv_freq, norm_rope64
from window_helpers import attend64, window_batch

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0


def place(cache, table, k, v, seq, pos):
    """Rows in their stored form at (seq, pos), by the append."""
    dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731
    cache.append(to_dev(k), to_dev(v), dev(seq), dev(pos), to_dev(table))


def moved(w, src_seq, src, dst_seq, dst, table=None, dst_table=None, **kw):
    """The workload's cache after the move."""
    cache, tab = device_cache(w, table=table, n_blocks=kw.pop("n_blocks", None))
    dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731
    cache.move_rows(dev(src_seq), dev(src), dev(dst_seq), dev(dst), tab, None if dst_table is None else to_dev(dst_table), **kw)
    return cache, tab


def first_rows(w):
    return np.concatenate([[0], np.cumsum(w.seq_lens)])


def check_bytes(w, src_seq, src, dst_seq, dst, table=None, dst_table=None, n_blocks=None, **kw):
    """Every byte of the pools: the moved rows at their places, all others as before."""
    cache, _ = moved(w, src_seq, src, dst_seq, dst, table, dst_table, n_blocks=n_blocks, **kw)
    want, _ = device_cache(w, table=table, n_blocks=n_blocks)
    row = first_rows(w)[np.asarray(src_seq)] + np.asarray(src)
    place(want, (w.table if table is None else table) if dst_table is None else dst_table, w.k_rows[row], w.v_rows[row], dst_seq, dst)
    torch.cuda.synchronize()
    assert cache.check() == PA_OK and want.check() == PA_OK
    assert torch.equal(cache.k_pool, want.k_pool) and torch.equal(cache.v_pool, want.v_pool)


PAIRS = [(F16, F16), (Q4, Q8), (Q8, Q4), (F16, Q4)]


@pytest.mark.parametrize("kt,vt", PAIRS)
@pytest.mark.parametrize("rows", [1, 5, 63, 64, 65, 256, 900])
@pytest.mark.parametrize("by", [1, 3, 16, 700])
def test_rows_moved_down_over_one_another(kt, vt, rows, by):
    """Few rows (one cluster) and many (through the workspace), by less than a row group and more."""
    w = window_batch([40, 1700], [1, 1], 48, kt, vt, seed=rows)
    check_bytes(w, [1] * rows, 4 + by + np.arange(rows), [1] * rows, 4 + np.arange(rows))


@pytest.mark.parametrize("rows", [30, 700])
def test_rows_reversed_swapped_and_kept(rows):
    """Every row's place is another's source, the middle one's its own; two sequences exchange theirs."""
    w = window_batch([800, 900], [1, 1], 16, Q8, Q4)
    at = np.arange(rows)
    check_bytes(w, [0] * rows, at, [0] * rows, at[::-1])
    seq = np.array([0] * (rows // 2) + [1] * (rows // 2))
    at = np.concatenate([np.arange(rows // 2)] * 2)
    check_bytes(w, seq, at, 1 - seq, at)


def test_copies_to_other_pages():
    """One row to many places, and rows through a table of their own with another stride."""
    w = window_batch([100, 64, 0], [1, 1, 0], 16, Q8, Q8)
    table = np.full((3, 20), -1, np.int32)
    table[:, : w.table.shape[1]] = w.table
    table[2, :9] = np.arange(w.n_blocks, w.n_blocks + 9)
    kw = dict(table=table, n_blocks=w.n_blocks + 20)
    check_bytes(w, [0] * 140, [33] * 140, [2] * 140, np.arange(140), disjoint=True, **kw)
    check_bytes(w, [0] * 140, [33] * 140, [2] * 140, np.arange(140), **kw)
    other = np.array([[w.n_blocks + 15, w.n_blocks + 12]], np.int32)
    check_bytes(w, [1] * 20, 10 + np.arange(20), [0] * 20, 5 + np.arange(20), dst_table=other, disjoint=True, **kw)
    check_bytes(w, [1] * 20, 10 + np.arange(20), [0] * 20, 5 + np.arange(20), dst_table=other, **kw)


@pytest.mark.parametrize("rows", [40, 700])
@pytest.mark.parametrize("disjoint", [False, True])
def test_rows_out_of_range_stay(rows, disjoint):
    w = window_batch([1000, 1000], [1, 1], 16, Q8, Q8)
    seq, src, dst_seq, dst = np.zeros(rows, int), np.arange(rows), np.ones(rows, int), np.arange(rows)
    good = np.ones(rows, bool)
    for i, (where, value) in enumerate([(seq, -1), (seq, 2), (src, -1), (src, 10 ** 6), (dst_seq, -1), (dst_seq, 9), (dst, -5), (dst, 2 ** 31 - 1)]):
        where[3 * i] = value
        good[3 * i] = False
    table = w.table.copy()
    table[1, 1] = w.n_blocks  # rows 16 .. 31 of the second sequence have no block
    good[16:32] = False
    cache, tab = device_cache(w)
    want = cache.k_pool.clone(), cache.v_pool.clone()
    dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731
    cache.move_rows(dev(seq), dev(src), dev(dst_seq), dev(dst), to_dev(table), disjoint=disjoint)
    assert cache.check() == PA_ERR_BOUNDS and cache.check() == PA_OK
    other = PagedKVCache(w.n_blocks, 16, Q8, Q8, k_pool=want[0], v_pool=want[1])
    place(other, w.table, w.k_rows[np.arange(rows)[good]], w.v_rows[np.arange(rows)[good]], np.ones(good.sum()), np.arange(rows)[good])
    assert other.check() == PA_OK
    assert torch.equal(cache.k_pool, other.k_pool) and torch.equal(cache.v_pool, other.v_pool)


def stored_within(got, want, mag, t, turned):
    """got: what a cache of this format gave back for values `want` (float64; mag: |a| + |b| of the pair behind each), where
    blocks were stored anew.  fp32 is off by 8 u mag (the cosine 5 u, its factor, product and sum a half step each), the format by
    half a step and the rounding of its scale (2^-11 of a value)."""
    u = 2.0 ** -24
    for b in range(8):
        if not turned[b]:
            assert np.array_equal(got[..., 32 * b: 32 * b + 32], want[..., 32 * b: 32 * b + 32])
            continue
        x, y = got[..., 32 * b: 32 * b + 32], want[..., 32 * b: 32 * b + 32]
        off = 8 * u * mag[..., 32 * b: 32 * b + 32].max(-1, keepdims=True)
        top = np.abs(y).max(-1, keepdims=True)
        if t == F16:
            bound = 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 2 * off
        elif t == Q8:  # a value of 127 steps at most
            bound = top / 127 * (0.5 + 127 * 2.0 ** -11) + 4 * off
        else:
            # 8 steps on the largest value's side, 7 (and a half step, then one cut off) on the other; where two of nearly one size and other
            # sign compete, either side may be it
            bound = top / 8 * (1.0 + 8 * 2.0 ** -11) + 4 * off
            inner = np.abs(y) <= 7.4 / 8 * top
            bound = np.where(inner, top / 8 * (0.5 + 8 * 2.0 ** -11) + 4 * off, bound)
        assert (np.abs(x - y) <= bound).all(), (t, b, (np.abs(x - y) / bound).max())


@pytest.mark.parametrize("kt", [F16, Q4, Q8])
@pytest.mark.parametrize("rot,inter", [(16, False), (32, True), (64, False), (80, False), (128, True), (256, False), (256, True)])
@pytest.mark.parametrize("rows,disjoint", [(50, False), (600, False), (600, True)])
def test_turned_keys(kt, rot, inter, rows, disjoint):
    """Keys at far positions moved to near ones; the first row keeps its position, and its bytes."""
    w = window_batch([20, 700], [1, 1], 16, kt, Q8, seed=rot)
    far = 3_000_000  # the position of the source table's first page
    table = np.full((1, far // 16 + w.table.shape[1]), -1, np.int32)
    table[0, far // 16:] = w.table[1]
    own = np.full((1, 200), -1, np.int32)
    own[0, :50] = w.n_blocks + np.random.default_rng(1).permutation(50)
    src, dst = far + 3 + np.arange(rows), 7 + np.arange(rows)
    f = inv_freq(rot, 1e7)
    cache, tab = device_cache(w, n_blocks=w.n_blocks + 50)
    dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731
    z = dev(np.zeros(rows))
    before = cache.k_pool.clone()
    cache.move_rows(z, dev(src), z, dev(dst), to_dev(table), to_dev(own), rope=Rope(f, interleaved=inter), disjoint=disjoint)
    k = torch.empty(rows, 4, 256, device="cuda")
    v = torch.empty(rows, 4, 256, device="cuda")
    cache.read_rows(z, dev(dst), to_dev(own), k_out=k, v_out=v)
    assert cache.check() == PA_OK
    at = 20 + 3 + np.arange(rows)
    x = oracle.dequant_rows(w.k_rows[at].reshape(rows * 4, -1), kt).reshape(rows, 4, 256)
    want, mag = norm_rope64(x, dst - src, f, inter)
    stored_within(k.cpu().numpy().astype(np.float64), want, mag, kt, [32 * b < rot for b in range(8)])
    assert np.array_equal(v.cpu().numpy(), oracle.dequant_rows(w.v_rows[at].reshape(rows * 4, -1), Q8).reshape(rows, 4, 256).astype(np.float32))
    # rows that stay where they are, turned by nothing
    cache.k_pool.copy_(before)
    cache.move_rows(z, dev(src), z, dev(src), to_dev(table), rope=Rope(f, interleaved=inter), disjoint=disjoint)
    assert cache.check() == PA_OK and torch.equal(cache.k_pool, before)


@pytest.mark.parametrize("kt", [F16, Q4, Q8])
@pytest.mark.parametrize("rows,disjoint", [(40, False), (600, False), (600, True)])
def test_frequencies_changed_in_place(kt, rows, disjoint):
    """From one set of frequencies and factor to another, each row where it lies."""
    w = window_batch([700], [1], 48, kt, Q8)
    old, new = Rope.from_theta(128, 1e6, attn_factor=1.25), Rope.scaled(128, 1e6, 4.0, "ramp", length=500, fast=8.0, attn_factor=1.1)
    cache, tab = device_cache(w)
    v0 = cache.v_pool.clone()
    dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731
    z, at = dev(np.zeros(rows)), dev(np.arange(rows))
    cache.move_rows(z, at, z, at, tab, rope=new, rope_from=old, disjoint=disjoint)
    k = torch.empty(700, 4, 256, device="cuda")
    cache.read_rows(dev(np.zeros(700)), dev(np.arange(700)), tab, k_out=k)
    assert cache.check() == PA_OK and torch.equal(cache.v_pool, v0)
    x = oracle.dequant_rows(w.k_rows.reshape(2800, -1), kt).reshape(700, 4, 256)
    delta = np.array(new.desc.inv_freq[:64]) - np.array(old.desc.inv_freq[:64])
    factor = new.desc.attn_factor / old.desc.attn_factor
    want, mag = norm_rope64(x[:rows], np.arange(rows), delta, factor=factor)
    got = k.cpu().numpy().astype(np.float64)
    stored_within(got[:rows], want, mag, kt, [b < 4 for b in range(8)])
    assert np.array_equal(got[rows:], x[rows:].astype(np.float32).astype(np.float64))


def test_heads_that_are_no_multiple_of_four():
    """A pool of six KV heads: few rows and many."""
    rng = np.random.default_rng(2)
    for rows in (20, 500):
        a, b = (PagedKVCache(80, 16, Q8, Q4, n_kv_heads=6) for _ in range(2))
        k, v = (to_dev(np.concatenate([W.random_rows(rng, 600, t), W.random_rows(rng, 600, t)[:, :2]], 1)) for t in (Q8, Q4))
        tab = torch.randperm(80, device="cuda").to(torch.int32)[:40][None]
        seq, at = torch.zeros(600, dtype=torch.int32, device="cuda"), torch.arange(600, dtype=torch.int32, device="cuda")
        for c in (a, b):
            c.append(k, v, seq, at, tab)
        a.move_rows(seq[:rows], at[:rows] + 30, seq[:rows], at[:rows], tab)
        b.append(k[30: 30 + rows].contiguous(), v[30: 30 + rows].contiguous(), seq[:rows], at[:rows], tab)
        assert a.check() == PA_OK and b.check() == PA_OK
        assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)


@pytest.mark.parametrize("kt,vt,page", [(F16, Q4, 16), (Q8, Q8, 64), (Q4, F16, 48), (Q8, Q4, 256)])
@pytest.mark.parametrize("n", [0, 1, 37, 150])
def test_blocks(kt, vt, page, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    nb = 400
    cache = PagedKVCache(nb, page, kt, vt)
    for pool in (cache.k_pool, cache.v_pool):
        pool.random_(0, 256, generator=g)
    order = torch.randperm(nb, device="cuda", generator=g).to(torch.int32)
    src, dst = order[:n].sort().values, order[n: 2 * n]
    table = torch.randint(-3, nb + 3, (7, 61), device="cuda", generator=g, dtype=torch.int32)
    table[0, :3] = torch.tensor([-2 ** 31, 2 ** 31 - 1, nb], device="cuda")
    want = [p.reshape(nb, -1).clone() for p in (cache.k_pool, cache.v_pool)]
    for p in want:
        p[dst.long()] = p[src.long()]
    to = {int(a): int(b) for a, b in zip(src, dst)}
    new = torch.tensor([[to.get(x, x) for x in row] for row in table.tolist()], dtype=torch.int32)
    before = table.clone()
    out = cache.move_blocks(src, dst, table)
    assert cache.check() == PA_OK
    assert torch.equal(out.cpu(), new) and torch.equal(table, before)
    assert all(torch.equal(p.reshape(nb, -1), q) for p, q in zip((cache.k_pool, cache.v_pool), want))
    assert cache.move_blocks(src, dst, table, table_out=table) is table and torch.equal(table.cpu(), new)
    assert cache.move_blocks(src, dst) is None and cache.check() == PA_OK
    assert all(torch.equal(p.reshape(nb, -1), q) for p, q in zip((cache.k_pool, cache.v_pool), want))


def test_blocks_out_of_range_and_out_of_order():
    cache = PagedKVCache(20, 16, Q8, Q8)
    cache.k_pool.random_(0, 256)
    want = cache.k_pool.clone().reshape(20, -1)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32(20, 3, 9)[None]
    out = cache.move_blocks(i32(3, 9, 20), i32(-1, 5, 6), table)  # neither place may be outside
    assert cache.check() == PA_ERR_BOUNDS
    want[5] = want[9]
    assert torch.equal(cache.k_pool.reshape(20, -1), want) and out.tolist() == [[20, 3, 5]]
    cache.move_blocks(i32(9, 3), i32(1, 2), table)
    assert cache.check() == PA_ERR_INVALID and cache.check() == PA_OK


def test_refusals():
    w = window_batch([100], [1], 16, Q8, Q8)
    cache, tab = device_cache(w)
    i = torch.arange(10, dtype=torch.int32, device="cuda")
    z = torch.zeros_like(i)
    good = dict(src_seq=z, src_pos=i, dst_seq=z, dst_pos=i, block_table=tab)
    before = cache.k_pool.clone()

    def refused(status=PA_ERR_INVALID, fn=cache.move_rows, **kw):
        with pytest.raises(PaError) as e:
            fn(**kw)
        assert e.value.status == status

    for kw in (dict(src_seq=z[:5]), dict(src_pos=i.long()), dict(dst_seq=z.cpu()), dict(dst_pos=i[::2]), dict(block_table=tab[0]),
               dict(dst_table=tab.long()), dict(rope_from=Rope(inv_freq(64))), dict(rope=Rope(inv_freq(64)), rope_from=Rope(inv_freq(32)))):
        refused(**{**good, **kw})
    refused(PA_ERR_UNSUPPORTED, **{**good, "rope": Rope(inv_freq(24))})
    many = torch.zeros(2000, dtype=torch.int32, device="cuda")
    refused(src_seq=many, src_pos=many, dst_seq=many, dst_pos=many, block_table=tab, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    blocks = dict(fn=cache.move_blocks, src=i[:2], dst=i[2:4], block_table=tab)
    for kw in (dict(src=i[:3]), dict(dst=i[2:4].long()), dict(block_table=tab.long()), dict(table_out=tab[:, :2].clone()),
               dict(block_table=None, table_out=tab)):
        refused(**{**blocks, **kw})
    torch.cuda.synchronize()
    assert cache.check() == PA_OK and torch.equal(cache.k_pool, before)


def test_captured_and_on_other_streams():
    """Captured and replayed on another state of the cache; on a stream passed in, with the arguments dropped at once."""
    w = window_batch([1700], [1], 16, Q8, Q8)
    rope = Rope(inv_freq(64))
    cache, tab = device_cache(w)
    k0, v0 = cache.k_pool.clone(), cache.v_pool.clone()
    for rows in (100, 900):
        z = torch.zeros(rows, dtype=torch.int32, device="cuda")
        at = torch.arange(rows, dtype=torch.int32, device="cuda")
        src = at + 333
        cache.k_pool.copy_(k0), cache.v_pool.copy_(v0)
        cache.move_rows(z, src, z, at, tab, rope=rope)
        want = cache.k_pool.clone(), cache.v_pool.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.move_rows(z, src, z, at, tab, rope=rope)
        side = torch.cuda.Stream()
        for how in ("replay", "stream", "replay"):
            cache.k_pool.copy_(k0), cache.v_pool.copy_(v0)
            if how == "replay":
                g.replay()
            else:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    torch.cuda._sleep(20_000_000)
                cache.move_rows(z.clone(), src.clone(), z.clone(), at.clone(), tab, rope=rope, stream=side)
                junk = [torch.full((rows,), 77, dtype=torch.int32, device="cuda") for _ in range(8)]
                side.synchronize()
                del junk
            torch.cuda.synchronize()
            assert cache.check() == PA_OK
            assert torch.equal(cache.k_pool, want[0]) and torch.equal(cache.v_pool, want[1])


def test_an_endless_conversation():
    """The operators together: a windowed sequence gives pages back, its pool is compacted, its
    context's middle is dropped with the later keys turned to their new positions, and the attention goes on."""
    rng = np.random.default_rng(8)
    kt, vt, page, window, sinks = F16, Q8, 16, 64, 4
    f = inv_freq(64, 1e4)
    rope = Rope(f)
    cache = PagedKVCache(40, page, kt, vt)
    pool = cache.pool
    # another sequence's pages leave holes
    other = pool.alloc(9)
    length = 300
    pages = pool.alloc(-(-length // page))
    assert pool.release(other) == PA_OK
    index = lambda hs: to_dev(np.array([[h & 0xffffffff for h in hs]], np.int32))  # noqa: E731
    raw = rng.standard_normal((length, 8, 256)).astype(np.float32)  # keys and values before the rotation
    x = to_dev(raw).half()
    at, z = torch.arange(length, dtype=torch.int32, device="cuda"), torch.zeros(length, dtype=torch.int32, device="cuda")
    cache.append_rope(rope, x[:, :4], x[:, 4:], z, at, index(pages))

    def attention(pos_of_rows, hs, n, w, s):
        """The newest n tokens' outputs, and what the stored rows at their positions should give."""
        m = len(pos_of_rows)
        q = rng.standard_normal((n, 24, 256)).astype(np.float32)
        lens = np.array([m], np.int32)
        out, _ = cache.attend_window(to_dev(q), index(hs), to_dev(lens), lens, np.array([n], np.int32), w, s)
        assert cache.check() == PA_OK
        half = x.cpu().numpy().astype(np.float64)[pos_of_rows]
        k, _ = norm_rope64(half[:, :4], np.arange(m), f)
        fake = W.Workload("", lens, 1, page, 1, kt, vt, np.zeros((1, 1), np.int32), np.zeros((1, 4, 512), np.uint8), np.zeros((1, 4, 272), np.uint8), q)
        want, _ = attend64(fake, [n], w, s, k=k, v=half[:, 4:])
        # Q8_0 values are off by half a step (|v| up to 4.5: 0.018) each, averaged by the weights; keys by binary16 roundings
        assert np.abs(out.cpu().numpy() - want).max() < 0.03

    attention(np.arange(length), pages, 3, window, sinks)
    # pages between sinks and window are given back
    keep = {0} | set(range((length - 3 - window + 1) // page, len(pages)))
    assert pool.release([h for i, h in enumerate(pages) if i not in keep]) == PA_OK
    free = pool.free_count()
    live = [h if i in keep else 0x7fffffff for i, h in enumerate(pages)]
    attention(np.arange(length), live, 3, window, sinks)
    # the pool is compacted
    moves = pool.compact()
    assert moves and pool.free_count() == free
    src, dst = (to_dev(np.array([m[i] & 0xffffffff for m in moves], np.int32)) for i in (0, 1))
    tab = cache.move_blocks(src, dst, index(live))
    live = [dict(moves).get(h, h) for h in live]
    assert torch.equal(tab, index(live))
    attention(np.arange(length), live, 3, window, sinks)
    # what is left becomes a short context: sinks, then the window's rows
    first = min(i for i in keep if i) * page
    rows = length - first
    n = to_dev(np.arange(first, length).astype(np.int32))
    to = to_dev((sinks + np.arange(rows)).astype(np.int32))
    # through a table in which the kept pages follow one another
    short = [live[i] for i in sorted(keep)]
    cache.move_rows(z[:rows], n, z[:rows], to, index(live), dst_table=index(short), rope=rope)
    assert cache.check() == PA_OK
    attention(np.concatenate([np.arange(sinks), np.arange(first, length)]), short, 5, 0, 0)
