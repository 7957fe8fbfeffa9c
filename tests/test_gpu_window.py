"""Attention over a sliding window and first keys against its definition in float64."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import assert_close, assert_lse_close, device_cache, to_dev
from paged_kv_gqa_11_gb300 import PA_ERR_BOUNDS, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_OK, PaError, pa_attend_window_workspace_size
from paged_kv_gqa_11_gb300.cache import PagedKVCache
from window_helpers import attend64, window_batch

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0


def attend(w, n_new, window, sinks, dtype=torch.float32, cache=None, tab=None, q=None, **kw):
    if cache is None:
        cache, tab = device_cache(w)
    q = to_dev(w.q).to(dtype) if q is None else q
    kw.setdefault("scale", w.scale)
    out, lse = cache.attend_window(q, tab, to_dev(w.seq_lens), w.seq_lens, np.asarray(n_new, np.int32), window, sinks, **kw)
    torch.cuda.synchronize()
    assert cache.check() == PA_OK
    return out, lse


def against_definition(w, n_new, window, sinks, dtype=torch.float32, what="", **kw):
    out, lse = attend(w, n_new, window, sinks, dtype, **kw)
    want, want_lse = attend64(w, n_new, window, sinks, to_dev(w.q).to(dtype).float().cpu().numpy())
    assert_close(out.float().cpu().numpy(), want, what=what)
    assert_lse_close(lse.cpu().numpy(), want_lse, what=what)


@pytest.mark.parametrize("kt", [F16, Q4, Q8])
@pytest.mark.parametrize("vt", [F16, Q4, Q8])
def test_every_format_pair(kt, vt):
    n_new = [1, 30, 2, 1]
    against_definition(window_batch([400, 333, 2, 150], n_new, 16, kt, vt), n_new, 100, 5, torch.float16)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 112, 113, 128, 129, 200, 256, 700, 1000, 5000, 0])
@pytest.mark.parametrize("sinks", [0, 1, 4, 16, 17, 130])
def test_windows_and_sinks(window, sinks):
    """Window and sinks that end at, before and after every tile, row group and page edge, that meet and overlap."""
    n_new = [1, 3, 1, 25, 1, 1]
    w = window_batch([700, 333, 1, 600, 129, 16], n_new, 48, Q8, Q4, seed=window + sinks)
    against_definition(w, n_new, window, sinks, torch.bfloat16, what=f"window {window}, sinks {sinks}")


@pytest.mark.parametrize("n", [1, 2, 3, 5, 10, 11, 12, 21, 22, 32, 33, 96, 97, 200])
def test_new_tokens(n):
    """Prompts from their first token on, chunks of longer ones, sequences without new tokens and empty ones."""
    n_new = [n, 0, n, 1, 0, max(1, n - 1)]
    w = window_batch([n, 50, n + 300, 1, 0, n + 77], n_new, 16, Q8, Q8, seed=n)
    against_definition(w, n_new, 70, 3, what=f"{n} tokens")
    against_definition(w, n_new, 0, 0, torch.float16, what=f"{n} tokens, no window")


@pytest.mark.parametrize("lens,n_new,window,sinks", [
    ([30000], [1], 0, 0), ([30000, 20, 9000], [1, 1, 1], 8192, 4), ([20000], [4], 0, 0), ([3000] * 20, [1] * 20, 1024, 16),
    ([5000, 700], [300, 1], 2048, 4), ([1500], [1500], 0, 0), ([40] * 130, [1] * 130, 32, 0)])
def test_pieces_of_many_ctas(lens, n_new, window, sinks):
    """Few long segments, cut by many CTAs, and many short ones, finished by one each."""
    against_definition(window_batch(lens, n_new, 64, Q4, Q8), n_new, window, sinks, torch.bfloat16)


def test_more_units_than_a_launch_takes():
    n_new = [1 + i % 3 for i in range(500)]
    lens = [n + (37 * i) % 90 for i, n in enumerate(n_new)]
    against_definition(window_batch(lens, n_new, 16, Q8, Q8), n_new, 40, 2, torch.float16)
    against_definition(window_batch([5300], [4900], 16, F16, F16), [4900], 60, 0, torch.float16)


@pytest.mark.parametrize("ot", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qt", [torch.float32, torch.float16, torch.bfloat16])
def test_types_strides_and_rows_behind_the_last_sequence(qt, ot):
    n_new = [1, 40, 2]
    w = window_batch([900, 500, 60], n_new, 32, Q8, Q4)
    cache, tab = device_cache(w)
    x = torch.full((50, 32, 256), float("nan"), device="cuda").to(qt)
    x[:43, :24] = to_dev(w.q).to(qt)
    big = torch.full((50, 30, 256), 7.0, device="cuda").to(ot)
    lse = torch.full((50, 24), 7.0, device="cuda")
    out, got = attend(w, n_new, 128, 4, cache=cache, tab=tab, q=x[:, :24], out=big[:, 3:27], lse=lse)
    assert got is lse and out.data_ptr() == big[:, 3:27].data_ptr()
    plain, plain_lse = attend(w, n_new, 128, 4, cache=cache, tab=tab, q=to_dev(w.q).to(qt), out=torch.empty(43, 24, 256, device="cuda"))
    assert torch.equal(out[:43], plain.to(ot)) and torch.equal(lse[:43], plain_lse)
    assert (out[43:] == 7).all() and (lse[43:] == 7).all() and (big[:, :3] == 7).all() and (big[:, 27:] == 7).all()
    out, lse = attend(w, n_new, 128, 4, cache=cache, tab=tab, q=x[:, :24])
    assert torch.equal(lse[:43], plain_lse) and (out[43:] == 0).all() and (lse[43:] == 0).all()
    out, lse = attend(w, n_new, 128, 4, cache=cache, tab=tab, q=x[:, :24], want_lse=False)
    assert lse is None and torch.equal(out[:43], plain.to(qt))


@pytest.mark.parametrize("kt,vt", [(F16, F16), (Q8, Q8), (Q4, Q4)])
@pytest.mark.parametrize("window,sinks", [(100, 0), (100, 5), (130, 40), (1, 0)])
def test_what_no_token_sees_has_no_effect(kt, vt, window, sinks):
    """Rows outside the windows that hold NaN and infinities, also in row groups that are read, and entries of
    released pages that lead nowhere."""
    n_new = [1, 20, 3]
    w = window_batch([1000, 777, 300], n_new, 16, kt, vt)
    cache, tab = device_cache(w)
    want, want_lse = attend(w, n_new, window, sinks, cache=cache, tab=tab)
    row, seen_pages = 0, []
    k, v = w.k_rows.copy(), w.v_rows.copy()
    for n, length in zip(n_new, w.seq_lens):
        x = np.arange(length)
        seen = (x > length - n - window) | (x < sinks)
        for rows, t in ((k, kt), (v, vt)):
            part = rows[row: row + length]
            part[~seen] = 0xff if t == F16 else part[~seen]
            if t != F16:  # scales that are infinite or NaN
                size = 34 if t == Q8 else 18
                for b in range(8):
                    part[~seen, :, size * b] = 0
                    part[~seen, :, size * b + 1] = 0x7c | (b & 1) << 1
            rows[row: row + length] = part
        seen_pages.append({int(p) // 16 for p in x[seen]})
        row += length
    bad = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, kt, vt, w.table, k, v, w.q, w.scale)
    cache, tab = device_cache(bad)
    holes = w.table.copy()
    for i, pages in enumerate(seen_pages):
        for p in range(holes.shape[1]):
            if p not in pages:
                holes[i, p] = [-1, 2 ** 31 - 1, w.n_blocks][p % 3]
    out, lse = attend(w, n_new, window, sinks, cache=cache, tab=to_dev(holes))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_bad_entries_and_lengths():
    n_new = [2, 1, 30, 1]
    w = window_batch([500, 300, 400, 90], n_new, 16, Q8, Q8)
    cache, tab = device_cache(w)
    want, want_lse = attend(w, n_new, 0, 0, cache=cache, tab=tab)
    lens = w.seq_lens.copy()
    lens[2] += 1
    q = to_dev(w.q)
    for window in (0, 20):  # cut among CTAs, and whole
        ref, ref_lse = attend(w, n_new, window, 0, cache=cache, tab=tab)
        out, lse = cache.attend_window(q, tab, to_dev(lens), w.seq_lens, np.array(n_new, np.int32), window, 0, w.scale)
        torch.cuda.synchronize()
        assert cache.check() == PA_ERR_BOUNDS and cache.check() == PA_OK
        other = torch.arange(34, device="cuda")[:, None].expand(34, 24)
        hit = (other >= 3) & (other < 33)
        assert (out[hit] == 0).all() and (lse[hit] == -float("inf")).all()
        assert torch.equal(out[~hit], ref[~hit]) and torch.equal(lse[~hit], ref_lse[~hit])
    holes = w.table.copy()
    holes[1, 3] = w.n_blocks  # 16 rows of zeros
    out, lse = cache.attend_window(q, to_dev(holes), to_dev(w.seq_lens), w.seq_lens, np.array(n_new, np.int32), 0, 0, w.scale)
    torch.cuda.synchronize()
    assert cache.check() == PA_ERR_BOUNDS
    k, v = w.k_rows.copy(), w.v_rows.copy()
    k[500 + 48: 500 + 64] = 0
    v[500 + 48: 500 + 64] = 0
    zero = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, Q8, w.table, k, v, w.q, w.scale)
    ref, ref_lse = attend64(zero, n_new, 0, 0)
    assert_close(out.cpu().numpy(), ref)
    assert_lse_close(lse.cpu().numpy(), ref_lse)


@pytest.mark.parametrize("size", [100.0, 60000.0])
def test_large_logits(size):
    """Windows whose later keys raise the reference by far, and whose first ones do."""
    n_new = [1, 15]
    w = window_batch([3000, 900], n_new, 16, F16, F16)
    k = W.encode_rows(np.sign(np.random.default_rng(1).standard_normal((3900, 4, 256))).astype(np.float32) * (size / 60000.0), F16)
    k[[2990, 2500, 3800, 3890]] = W.encode_rows(np.full((4, 4, 256), size / 2000.0, np.float32), F16)
    w = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, F16, F16, w.table, k, w.v_rows, np.abs(w.q), w.scale)
    against_definition(w, n_new, 600, 4, torch.float16)
    against_definition(w, n_new, 0, 0, torch.float16)


def test_equals_the_decode_without_a_window():
    w = W.small_workload(5, [300, 900, 41], 16, Q8)
    cache, tab = device_cache(w)
    want, want_lse = cache.decode(to_dev(w.q), tab, to_dev(w.seq_lens), w.seq_lens, w.n_qtok, w.scale)
    out, lse = cache.attend_window(to_dev(w.q).reshape(-1, 24, 256), tab, to_dev(w.seq_lens), w.seq_lens,
                                   np.full(len(w.seq_lens), w.n_qtok, np.int32), scale=w.scale)
    assert cache.check() == PA_OK
    assert_close(out.reshape(want.shape).cpu().numpy(), want.cpu().numpy().astype(np.float64))
    assert_lse_close(lse.reshape(want_lse.shape).cpu().numpy(), want_lse.cpu().numpy())


def test_streams_graphs_and_repeats():
    """The same call gives the same bits: again, on two other streams at once, captured and replayed with other queries, with
    the caller's workspace."""
    n_new = [1, 60, 4]
    w = window_batch([4000, 2500, 900], n_new, 16, Q8, Q4)
    cache, tab = device_cache(w)
    q, sl, nn = to_dev(w.q).half(), to_dev(w.seq_lens), np.array(n_new, np.int32)
    call = lambda q, **kw: cache.attend_window(q, tab, sl, w.seq_lens, nn, 1500, 4, w.scale, **kw)  # noqa: E731
    want, want_lse = call(q)
    q2 = q.flip(0).contiguous()
    want2, _ = call(q2)
    ws = torch.full((pa_attend_window_workspace_size(cache.pool, w.seq_lens, n_new, 1500, 4),), 255, dtype=torch.uint8, device="cuda")
    got, got_lse = call(q, workspace=ws)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    res = []
    for i in range(6):
        res.append((i, call(q2 if i % 2 else q, stream=streams[i % 2])[0]))
    torch.cuda.synchronize()
    for i, r in res:
        assert torch.equal(r, want2 if i % 2 else want)
    g = torch.cuda.CUDAGraph()
    x = q.clone()
    with torch.cuda.graph(g):
        y, _ = call(x)
    for src, ref in ((q, want), (q2, want2), (q, want)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    assert cache.check() == PA_OK


def test_refusals():
    w = window_batch([100, 50], [3, 1], 16, Q8, Q8)
    cache, tab = device_cache(w)
    q, sl, nn = to_dev(w.q), to_dev(w.seq_lens), np.array([3, 1], np.int32)
    good = dict(q=q, block_table=tab, seq_lens_dev=sl, seq_lens_host=w.seq_lens, n_new=nn)

    def refused(status=PA_ERR_INVALID, **kw):
        with pytest.raises(PaError) as e:
            cache.attend_window(**{**good, **kw})
        assert e.value.status == status

    refused(q=q[:3])
    refused(q=q.cpu())
    refused(q=q[:, :18], status=PA_ERR_UNSUPPORTED)
    refused(q=q[..., :128])
    refused(q=q.double(), status=PA_ERR_UNSUPPORTED)
    refused(q=q.transpose(0, 1))
    refused(n_new=np.array([3, -1], np.int32))
    refused(n_new=np.array([3], np.int32))
    refused(n_new=np.array([3, 1], np.int64))
    refused(n_new=np.array([3, 51], np.int32), q=torch.zeros(54, 24, 256, device="cuda"))
    refused(seq_lens_host=np.array([100, 200], np.int32))
    refused(window=-1)
    refused(sinks=-1)
    refused(window=2 ** 32)
    refused(scale=0.0)
    refused(scale=float("nan"))
    refused(out=torch.empty(4, 24, 128, device="cuda"))
    refused(out=torch.empty(5, 24, 256, device="cuda"))
    refused(out=torch.empty(24, 4, 256, device="cuda").transpose(0, 1))
    refused(lse=torch.empty(4, 24, dtype=torch.float16, device="cuda"))
    refused(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    refused(block_table=tab[:1])
    refused(seq_lens_dev=sl.long())
    out, lse = cache.attend_window(**{**good, "n_new": np.zeros(2, np.int32)})
    assert (out == 0).all() and (lse == 0).all()
    torch.cuda.synchronize()
    assert cache.check() == PA_OK
    PagedKVCache(1, 16, Q8, Q8)


@pytest.mark.parametrize("kt,vt", [(F16, F16), (Q4, Q8), (Q8, Q4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 1), (100, 4), (128, 16), (129, 130), (600, 17), (2000, 0)])
def test_prompts(kt, vt, window, sinks):
    """Sequences of many new tokens beside those of few: from the first token on, after others, of odd lengths, with
    pages that no power of two counts."""
    n_new = [64, 1, 150, 0, 300, 63, 65]
    lens = [64, 700, 151, 0, 1100, 63, 1500]
    w = window_batch(lens, n_new, 48, kt, vt, seed=window + sinks)
    against_definition(w, n_new, window, sinks, torch.bfloat16, what=f"window {window}, sinks {sinks}")


@pytest.mark.parametrize("qt,ot", [(torch.float32, torch.float16), (torch.float16, torch.float32), (torch.bfloat16, torch.bfloat16)])
def test_prompts_in_rows_of_any_type(qt, ot):
    n_new = [70, 90]
    w = window_batch([500, 90], n_new, 16, Q8, Q8)
    x = torch.full((170, 32, 256), float("nan"), device="cuda").to(qt)
    x[:160, :24] = to_dev(w.q).to(qt)
    big = torch.full((170, 30, 256), 7.0, device="cuda").to(ot)
    lse = torch.full((170, 24), 7.0, device="cuda")
    cache, tab = device_cache(w)
    out, _ = attend(w, n_new, 128, 4, cache=cache, tab=tab, q=x[:, :24], out=big[:, 3:27], lse=lse)
    want, want_lse = attend64(w, n_new, 128, 4, x[:160, :24].float().cpu().numpy())
    assert_close(out[:160].float().cpu().numpy(), want)
    assert_lse_close(lse[:160].cpu().numpy(), want_lse)
    assert (out[160:] == 7).all() and (lse[160:] == 7).all() and (big[:, :3] == 7).all() and (big[:, 27:] == 7).all()


def test_prompts_of_one_launch_and_several():
    against_definition(window_batch([6000], [5800], 64, Q8, Q8), [5800], 80, 4, torch.float16)  # more than 256 units
    n_new = [64 + i % 3 for i in range(140)]  # more sequences than a launch prepares
    against_definition(window_batch([n + 5 * (i % 7) for i, n in enumerate(n_new)], n_new, 16, F16, F16), n_new, 0, 0, torch.float16)
    against_definition(window_batch([12000], [64], 16, Q4, Q4), [64], 0, 0, torch.bfloat16)  # long segments, cut by many CTAs


@pytest.mark.parametrize("size", [100.0, 60000.0])
def test_prompts_with_large_logits(size):
    """Later keys that raise the reference by far."""
    n_new = [200]
    w = window_batch([900], n_new, 16, F16, F16)
    k = W.encode_rows(np.sign(np.random.default_rng(1).standard_normal((900, 4, 256))).astype(np.float32) * (size / 60000.0), F16)
    k[[3, 650, 790, 890]] = W.encode_rows(np.full((4, 4, 256), size / 2000.0, np.float32), F16)
    w = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, F16, F16, w.table, k, w.v_rows, np.abs(w.q), w.scale)
    against_definition(w, n_new, 600, 4, torch.float16)
    against_definition(w, n_new, 0, 0, torch.float16)


@pytest.mark.parametrize("kt", [Q4, Q8])
@pytest.mark.parametrize("n", [3, 80])
def test_stored_keys_past_binary16(kt, n):
    """Scales times quants of up to 8.3 10^6 in a few keys, whose logits the small queries keep in range."""
    n_new = [n]
    w = window_batch([400], n_new, 16, kt, Q8)
    k = w.k_rows.copy()
    size = 34 if kt == Q8 else 18
    for row in (0, 7, 130, 200, 399):
        scales = k[row].reshape(4, 8, size)[..., :2].copy().view(np.float16)
        k[row].reshape(4, 8, size)[..., :2] = (scales / np.abs(scales).max() * 60000).astype(np.float16).view(np.uint8).reshape(4, 8, 2)
    w = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, kt, Q8, w.table, k, w.v_rows, (w.q * 1e-5).astype(np.float32), w.scale)
    # queries this small are subnormal in binary16: powers of two keep them exact
    q = np.sign(w.q).astype(np.float32) * 2.0 ** -20
    w = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, kt, Q8, w.table, k, w.v_rows, q, w.scale)
    against_definition(w, n_new, 300, 4)
    against_definition(w, n_new, 0, 0)


@pytest.mark.parametrize("kt,vt", [(F16, F16), (Q8, Q4)])
def test_prompts_and_what_no_token_sees(kt, vt):
    """Rows before the windows and behind the sequences, in row groups that are read, that hold NaN and infinities."""
    n_new, window, sinks = [100, 64], 60, 5
    w = window_batch([1000, 333], n_new, 16, kt, vt)
    cache, tab = device_cache(w)
    want, want_lse = attend(w, n_new, window, sinks, cache=cache, tab=tab)
    row = 0
    k, v = w.k_rows.copy(), w.v_rows.copy()
    for n, length in zip(n_new, w.seq_lens):
        x = np.arange(length)
        dead = ~((x > length - n - window) | (x < sinks))
        for rows, t in ((k, kt), (v, vt)):
            part = rows[row: row + length]
            if t == F16:
                part[dead] = 0xff
            else:
                size = 34 if t == Q8 else 18
                for b in range(8):
                    part[dead, :, size * b] = 0
                    part[dead, :, size * b + 1] = 0x7c | (b & 1) << 1
        row += length
    bad = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, kt, vt, w.table, k, v, w.q, w.scale)
    cache, tab = device_cache(bad)
    # the last pages' other rows too
    for i, length in enumerate(w.seq_lens):
        rest = np.arange(length, -(-int(length) // 16) * 16)
        nan = lambda t: np.full((len(rest), 4, W.row_bytes(t)), 0xff, np.uint8)  # noqa: E731
        dev = lambda x: to_dev(np.ascontiguousarray(x, dtype=np.int32))  # noqa: E731
        if len(rest):
            cache.append(to_dev(nan(kt)), to_dev(nan(vt)), dev(np.full(len(rest), i)), dev(rest), tab)
    out, lse = attend(w, n_new, window, sinks, cache=cache, tab=tab)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_prompts_with_bad_entries_and_lengths():
    n_new = [100, 1, 64]
    w = window_batch([500, 300, 400], n_new, 16, Q8, Q8)
    cache, tab = device_cache(w)
    lens = w.seq_lens.copy()
    lens[0] -= 1
    q = to_dev(w.q)
    for window in (0, 50):
        ref, ref_lse = attend(w, n_new, window, 0, cache=cache, tab=tab)
        out, lse = cache.attend_window(q, tab, to_dev(lens), w.seq_lens, np.array(n_new, np.int32), window, 0, w.scale)
        torch.cuda.synchronize()
        assert cache.check() == PA_ERR_BOUNDS and cache.check() == PA_OK
        assert (out[:100] == 0).all() and (lse[:100] == -float("inf")).all()
        assert torch.equal(out[100:], ref[100:]) and torch.equal(lse[100:], ref_lse[100:])
    holes = w.table.copy()
    holes[2, 3] = -7  # 16 rows of zeros
    out, lse = cache.attend_window(q, to_dev(holes), to_dev(w.seq_lens), w.seq_lens, np.array(n_new, np.int32), 0, 0, w.scale)
    torch.cuda.synchronize()
    assert cache.check() == PA_ERR_BOUNDS
    k, v = w.k_rows.copy(), w.v_rows.copy()
    k[800 + 48: 800 + 64] = 0
    v[800 + 48: 800 + 64] = 0
    zero = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, Q8, w.table, k, v, w.q, w.scale)
    ref, ref_lse = attend64(zero, n_new, 0, 0)
    assert_close(out.cpu().numpy(), ref)
    assert_lse_close(lse.cpu().numpy(), ref_lse)


def test_prompts_repeat_bit_for_bit():
    """Again, captured and replayed with other queries, on another stream at once."""
    n_new = [300, 80, 1]
    w = window_batch([2500, 900, 77], n_new, 16, Q8, Q4)
    cache, tab = device_cache(w)
    q, sl, nn = to_dev(w.q).half(), to_dev(w.seq_lens), np.array(n_new, np.int32)
    call = lambda q, **kw: cache.attend_window(q, tab, sl, w.seq_lens, nn, 1500, 4, w.scale, **kw)  # noqa: E731
    q2 = q.flip(0).contiguous()
    want, want2 = call(q)[0], call(q2)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    res = [(i, call(q2 if i % 2 else q, stream=side if i % 2 else None)[0]) for i in range(6)]
    g = torch.cuda.CUDAGraph()
    x = q.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y, _ = call(x)
    for i, r in res:
        assert torch.equal(r, want2 if i % 2 else want)
    for src, ref in ((q, want), (q2, want2), (q, want)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    assert cache.check() == PA_OK


# One new token per sequence in batches that fill the device, K Q8_0: clusters of 1, 2, 4 and 8 CTAs, several waves and launches.
STEPS = [(64, 1, 0), (64, 16, 1), (64, 17, 0), (70, 64, 5), (76, 100, 16), (61, 33, 40), (64, 1000, 130), (33, 500, 4), (16, 600, 17),
         (8, 1030, 0), (8, 1500, 3), (300, 540, 3)]


def step_batch(seqs, window, sinks, vt, seed=1, ps=48):
    """Sequences longer than the window by less than it takes for one to stand out, and one without a new token."""
    lens = [max(1, window) + sinks + (37 * i) % 90 for i in range(seqs)]
    return window_batch(lens + [20], [1] * seqs + [0], ps, Q8, vt, seed=seed), [1] * seqs + [0]


@pytest.mark.parametrize("vt", [Q4, Q8])
@pytest.mark.parametrize("seqs,window,sinks", STEPS)
def test_steps(seqs, window, sinks, vt):
    w, n_new = step_batch(seqs, window, sinks, vt, seed=seqs + window)
    against_definition(w, n_new, window, sinks, torch.bfloat16 if vt == Q4 else torch.float16, what=f"{seqs} x {window}, {sinks}")


def test_steps_without_a_window():
    """Idle sequences between the others, lengths from 60 to 70."""
    n_new = [i % 5 != 3 for i in range(85)]
    w = window_batch([60 + i % 11 for i in range(85)], n_new, 16, Q8, Q8)
    against_definition(w, n_new, 0, 0)
    w = window_batch([1] * 64, [1] * 64, 16, Q8, Q4)
    against_definition(w, [1] * 64, 0, 0, torch.float16)


def test_steps_beside_prompts():
    """Single tokens by their kernel, chunks of prompt between them by theirs."""
    n_new = [1] * 20 + [100] + [1] * 30 + [0, 64] + [1] * 14
    w = window_batch([150 + i % 9 for i in range(len(n_new))], n_new, 16, Q8, Q8)
    against_definition(w, n_new, 90, 3, torch.float16)
    n_new = [200] + [1] * 300
    w = window_batch([600 if i == 0 else 560 + i % 9 for i in range(301)], n_new, 32, Q8, Q4)
    against_definition(w, n_new, 540, 0, torch.bfloat16)


@pytest.mark.parametrize("ot", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("seqs", [64, 16])
def test_steps_types_strides_and_rows_behind_the_last_sequence(seqs, qt, ot):
    w, n_new = step_batch(seqs, 700, 4, Q4)
    cache, tab = device_cache(w)
    x = torch.full((seqs + 5, 32, 256), float("nan"), device="cuda").to(qt)
    x[:seqs, :24] = to_dev(w.q).to(qt)
    big = torch.full((seqs + 5, 30, 256), 7.0, device="cuda").to(ot)
    lse = torch.full((seqs + 5, 24), 7.0, device="cuda")
    out, _ = attend(w, n_new, 700, 4, cache=cache, tab=tab, q=x[:, :24], out=big[:, 3:27], lse=lse)
    plain, plain_lse = attend(w, n_new, 700, 4, cache=cache, tab=tab, q=to_dev(w.q).to(qt), out=torch.empty(seqs, 24, 256, device="cuda"))
    assert torch.equal(out[:seqs], plain.to(ot)) and torch.equal(lse[:seqs], plain_lse)
    assert (out[seqs:] == 7).all() and (lse[seqs:] == 7).all() and (big[:, :3] == 7).all() and (big[:, 27:] == 7).all()


@pytest.mark.parametrize("seqs,window,sinks", [(64, 100, 5), (33, 301, 0), (16, 600, 17), (64, 1, 0)])
@pytest.mark.parametrize("vt", [Q4, Q8])
def test_steps_and_what_no_token_sees(seqs, window, sinks, vt):
    w, n_new = step_batch(seqs, window, sinks, vt, ps=16)
    cache, tab = device_cache(w)
    want, want_lse = attend(w, n_new, window, sinks, cache=cache, tab=tab)
    k, v = w.k_rows.copy(), w.v_rows.copy()
    holes, row = w.table.copy(), 0
    for i, length in enumerate(w.seq_lens):
        x = np.arange(length)
        unseen = ~((x >= length - window) | (x < sinks)) if n_new[i] else x >= 0
        for rows, size in ((k, 34), (v, 34 if vt == Q8 else 18)):
            part = rows[row: row + length]
            for b in range(8):  # scales that are infinite or NaN
                part[unseen, :, size * b] = 0
                part[unseen, :, size * b + 1] = 0x7c | (b & 1) << 1
        seen_pages = {int(p) // 16 for p in x[~unseen]}
        for p in range(holes.shape[1]):
            if p not in seen_pages:
                holes[i, p] = [-1, 2 ** 31 - 1, w.n_blocks][p % 3]
        row += length
    bad = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, vt, w.table, k, v, w.q, w.scale)
    cache, _ = device_cache(bad)
    out, lse = attend(w, n_new, window, sinks, cache=cache, tab=to_dev(holes))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("seqs,window", [(64, 150), (16, 600)])
def test_steps_with_bad_entries_and_lengths(seqs, window):
    w, n_new = step_batch(seqs, window, 0, Q8, ps=16)
    cache, tab = device_cache(w)
    want, want_lse = attend(w, n_new, window, 0, cache=cache, tab=tab)
    lens, nn, q = w.seq_lens.copy(), np.array(n_new, np.int32), to_dev(w.q)
    lens[5] -= 1
    out, lse = cache.attend_window(q, tab, to_dev(lens), w.seq_lens, nn, window, 0, w.scale)
    torch.cuda.synchronize()
    assert cache.check() == PA_ERR_BOUNDS and cache.check() == PA_OK
    keep = torch.arange(seqs, device="cuda") != 5
    assert (out[5] == 0).all() and (lse[5] == -float("inf")).all()
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    for entry in (-1, w.n_blocks, 2 ** 31 - 1):
        holes = w.table.copy()
        page = int(w.seq_lens[7] - 40) // 16
        holes[7, page] = entry  # 16 rows of zeros
        out, lse = cache.attend_window(q, to_dev(holes), to_dev(w.seq_lens), w.seq_lens, nn, window, 0, w.scale)
        torch.cuda.synchronize()
        assert cache.check() == PA_ERR_BOUNDS and cache.check() == PA_OK
        k, v = w.k_rows.copy(), w.v_rows.copy()
        at = int(w.seq_lens[:7].sum()) + 16 * page
        k[at: at + 16] = 0
        v[at: at + 16] = 0
        zero = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, Q8, w.table, k, v, w.q, w.scale)
        ref, ref_lse = attend64(zero, n_new, window, 0)
        assert_close(out.cpu().numpy(), ref)
        assert_lse_close(lse.cpu().numpy(), ref_lse)


@pytest.mark.parametrize("seqs,window", [(64, 300), (16, 600)])
@pytest.mark.parametrize("size", [100.0, 60000.0])
def test_steps_with_large_logits(seqs, window, size):
    """Later keys that raise a warp's reference until what came before is nothing, very negative first ones, keys past binary16."""
    w, n_new = step_batch(seqs, window, 4, Q4, ps=16)
    rng = np.random.default_rng(4)
    x = np.sign(rng.standard_normal((len(w.k_rows), 4, 256))).astype(np.float32) * (size / 60000.0)
    ends = np.cumsum(w.seq_lens)
    for s in range(seqs):  # one large key somewhere in the window, in others all but it very negative
        at = ends[s] - 1 - (s * 29) % window
        if s % 3 == 2:
            x[ends[s] - w.seq_lens[s]: ends[s]] = -size / 2000.0
        x[at] = size / 2000.0
    k = W.encode_rows(x, Q8)
    w = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, Q4, w.table, k, w.v_rows, np.abs(w.q), w.scale)
    against_definition(w, n_new, window, 4, torch.float16)
    scales = k.reshape(len(k), 4, 8, 34)[..., :2].copy().view(np.float16)
    scales[:] = 60000  # quants up to 127: keys of 7.6 10^6
    k.reshape(len(k), 4, 8, 34)[..., :2] = scales.view(np.uint8).reshape(len(k), 4, 8, 2)
    q = np.sign(w.q).astype(np.float32) * 2.0 ** -20
    w = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, Q4, w.table, k, w.v_rows, q, w.scale)
    against_definition(w, n_new, window, 4)


def test_steps_past_the_queries_range():
    """Queries past binary16's range give NaN in their rows, and there alone."""
    w, n_new = step_batch(64, 100, 0, Q8)
    cache, tab = device_cache(w)
    q = to_dev(w.q).clone()
    want, want_lse = attend(w, n_new, 100, 0, cache=cache, tab=tab, q=q)
    q[3, 7, 200] = 70000.0
    q[3, 23, 1] = float("inf")
    q[60, 0, 255] = float("nan")
    out, lse = attend(w, n_new, 100, 0, cache=cache, tab=tab, q=q)
    hit = torch.zeros(64, 24, dtype=torch.bool, device="cuda")
    hit[3, 7] = hit[3, 23] = hit[60, 0] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])


def test_steps_streams_graphs_and_repeats():
    w, n_new = step_batch(33, 600, 4, Q4)
    cache, tab = device_cache(w)
    q, sl, nn = to_dev(w.q).half(), to_dev(w.seq_lens), np.array(n_new, np.int32)
    call = lambda q, **kw: cache.attend_window(q, tab, sl, w.seq_lens, nn, 600, 4, w.scale, **kw)  # noqa: E731
    want, want_lse = call(q)
    q2 = q.flip(0).contiguous()
    want2, _ = call(q2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    res = [(i, call(q2 if i % 2 else q, stream=streams[i % 2])[0]) for i in range(6)]
    torch.cuda.synchronize()
    for i, r in res:
        assert torch.equal(r, want2 if i % 2 else want)
    g = torch.cuda.CUDAGraph()
    x = q.clone()
    with torch.cuda.graph(g):
        y, _ = call(x)
    for src, ref in ((q, want), (q2, want2), (q, want)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    assert cache.check() == PA_OK
