"""Shared-prefix decode at the edges of its number types: what is not finite
shows in the outputs, and stored keys of any size count as what they are."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import assert_close, assert_lse_close, device_cache, to_dev
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


# ------------------------------------------------------------------ the range of stored keys

def attend64(w, k, v, q):
    """The definition in float64 on given rows [n][heads][256] (stored order) -> (out, lse, max of scale sum |q||k|)."""
    out, lse, at, most = np.zeros(w.q.shape), np.zeros(w.q.shape[:3]), 0, 0.0
    t = w.n_qtok
    for s, n in enumerate(w.seq_lens.tolist()):
        for h in range(24):
            kh, vh = k[at:at + n, h // 6], v[at:at + n, h // 6]
            for i in range(t):
                m = n - t + 1 + i
                z = w.scale * (kh[:m] @ q[s, i, h])
                most = max(most, w.scale * (np.abs(kh[:m]) @ np.abs(q[s, i, h])).max())
                p = np.exp(z - z.max())
                lse[s, i, h] = z.max() + np.log(p.sum())
                out[s, i, h] = p @ vh[:m] / p.sum()
        at += n
    return out, lse, most


def wide_keys(w, kt, every, seed):
    """w with K rows encoded anew: dims 64 .. 95 of every `every`-th row are about 5 * 10^4 N(0, 1) (past binary16's range, in scales within it), with
    queries of about 10^-5 there, so that the logits stay ordinary."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((len(w.k_rows), 4, 256)).astype(np.float32)
    pos = np.concatenate([np.arange(n) for n in w.seq_lens])
    x = x[np.minimum(pos, len(x) - 1)]  # rows by position: the prefix's copies are alike
    x[pos % every == 0, :, 64:96] *= np.float32(5e4)
    q = w.q.copy()
    q[..., 64:96] *= np.float32(1e-5)
    return W.Workload(w.name, w.seq_lens, w.n_qtok, w.page_size, w.n_blocks, kt, w.v_type, w.table, W.encode_rows(x, kt), w.v_rows, q, w.scale)


@pytest.mark.parametrize("kt", [Q8, Q4])
@pytest.mark.parametrize("t", [1, 4])
@pytest.mark.parametrize("every", [1, 7, 901])
def test_keys_past_binary16(kt, t, every):
    """Scale * quant past 65504: finite in the pool, and the product with a small
    query an ordinary logit -- every key so, some of them, a few."""
    w, gs, pl = prefix_workload([(3, 1500), (1, 20)], [200, 40, 1000, 30], 16, kt, Q8, n_qtok=t)
    w = wide_keys(w, kt, every, seed=t)
    q = to_dev(w.q).half()
    out, lse = decode(w, gs, pl, q)
    k, v = oracle.dequant_rows(w.k_rows, kt), oracle.dequant_rows(w.v_rows, Q8)
    assert np.abs(k).max() > 65504
    want, want_lse, _ = attend64(w, k, v, q.double().cpu().numpy())
    assert_close(out.cpu().numpy(), want)
    assert_lse_close(lse.cpu().numpy(), want_lse)


def test_wide_keys_leave_the_others_alone():
    """A sequence with such keys in a batch changes no bit of the other sequences."""
    w, gs, pl = prefix_workload([(2, 700), (3, 500)], [100, 40, 300, 30, 60], 16, Q8, Q8)
    q = to_dev(w.q).half()
    want, want_lse = decode(w, gs, pl, q)
    k = w.k_rows.copy().reshape(len(w.k_rows), 4, 8, 34)
    at = int(w.seq_lens[:4].sum()) + 520  # the fifth sequence's own row
    k[at, :, 3, :2] = np.array([3000.0], np.float16).view(np.uint8)
    bad = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, Q8, w.table, k.reshape(w.k_rows.shape), w.v_rows, w.q, w.scale)
    out, lse = decode(bad, gs, pl, q)
    assert torch.equal(out[:4], want[:4]) and torch.equal(lse[:4], want_lse[:4])
    kd, vd = oracle.dequant_rows(bad.k_rows, Q8), oracle.dequant_rows(w.v_rows, Q8)
    ref, ref_lse, _ = attend64(bad, kd, vd, q.double().cpu().numpy())
    # the key's logits are tens of thousands: a row sees it alone or not at all (2^-11 of |q||k| scale is some tens)
    z = np.abs(np.einsum("hgd,hd->hg", q[4, 0].double().cpu().numpy().reshape(4, 6, 256), kd[at]).reshape(24)) / 16
    sharp = z > 500
    assert sharp.sum() > 20
    assert_close(out.cpu().numpy()[4, 0][sharp], ref[4, 0][sharp])
    assert (np.abs(lse.cpu().numpy() - ref_lse)[4, 0] <= 2.0 ** -11 * 16 * z + 0.01).all()


# ------------------------------------------------------------------ the range of queries

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [1e5, -3e38, 65536.0])
@pytest.mark.parametrize("kt", [F16, Q4])
def test_queries_past_binary16_are_not_a_number(dtype, value, kt):
    """A finite query value that binary16 has no number for makes its row NaN, whatever
    the keys' signs; the other rows stay as they are."""
    w, gs, pl = prefix_workload([(4, 2000), (1, 30)], [40, 50, 30, 400, 20], 16, kt, Q8)
    if kt == F16:  # all of a dim's keys of one sign: every logit would be -inf or inf
        k = np.ascontiguousarray(w.k_rows).view(np.float16).copy()
        k[..., 9] = np.abs(k[..., 9]) + np.float16(0.125)
        w = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, kt, Q8, w.table, k.view(np.uint8), w.v_rows, w.q, w.scale)
    q = to_dev(w.q).to(dtype)
    want, want_lse = decode(w, gs, pl, q)
    q[2, 0, 23, 9] = value
    out, lse = decode(w, gs, pl, q)
    mark = torch.zeros(5, 1, 24, dtype=torch.bool, device="cuda")
    mark[2, 0, 23] = True
    assert out[mark].isnan().all() and lse[mark].isnan().all()
    assert torch.equal(out[~mark], want[~mark]) and torch.equal(lse[~mark], want_lse[~mark])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_queries(dtype):
    """Just inside the range (65280 has a bfloat16): an ordinary row."""
    w, gs, pl = prefix_workload([(3, 600)], [40, 50, 30], 16, Q8, Q8)
    q = to_dev(w.q).to(dtype)
    q[1, 0, 5, :] = 0
    q[1, 0, 5, 200] = 65280.0
    out, lse = decode(w, gs, pl, q)
    assert out.isfinite().all() and lse.isfinite().all()


# ------------------------------------------------------------------ precision

def bounds(w, k, v, q, want, key_step):
    """How far out and lse may lie from `want`, the float64 result on the rows k and v
    (per element of out; one number for lse).

    Logits: products of binary16 numbers are exact in fp32; the sum over 256 dims is 16
    steps of 16 dims, each off by 2^-23 of sum |q||k| at most; scale (its conversion to log2
    units), the difference from the reference and ex2 are off by 2^-21 of the logit and
    2^-21 -- d below -- and the stored keys' own rounding by key_step * scale sum |q||k|.
    Weights p e^(+-d), renormalised: off by e^(2 d) - 1 relative.  The weights' rounding
    (2^-11, or half of 2^-24 for weights below 2^-14, against a sum of 1 at least) and V's
    (2^-11) come on top."""
    out, lse, most = want
    absolute, _, _ = attend64(w, k, np.abs(v), q)
    d = (2.0 ** -19 + 2.0 ** -21 + key_step) * most + 2.0 ** -21
    few = w.seq_lens.max() * 2.0 ** -25 * np.abs(v).max()
    return (np.expm1(2 * d) + 2.0 ** -10 * 1.01) * (absolute + np.abs(out)) + few, d + 2.0 ** -11 + 2.0 ** -22 * np.abs(lse).max()


@pytest.mark.parametrize("kt,vt", [(Q8, Q4), (Q4, Q8), (F16, F16)])
@pytest.mark.parametrize("t", [1, 4])
def test_large_logits(kt, vt, t):
    """Logits of standard deviation 16.  Against the keys as they are: within the stated
    2^-11 |q||k| scale of every logit.  Against the keys rounded to binary16: within the
    rounding of the rest, so that nothing but the stated rounding is lost."""
    base = W.stress_workload("bigq", 77, [2000], 16, kt, vt, t)
    n, rows, pages = 2000, 1008, 125
    table = np.stack([np.arange(pages), np.concatenate([np.arange(rows // 16), pages + np.arange(pages - rows // 16)])]).astype(np.int32)
    w = W.Workload("bigq", np.array([n, n], np.int32), t, 16, 2 * pages, kt, vt, table, np.concatenate([base.k_rows] * 2),
                   np.concatenate([base.v_rows] * 2), np.concatenate([base.q, base.q]), base.scale)
    out, lse = decode(w, np.array([2], np.uint32), np.array([rows], np.int32), to_dev(w.q).half())
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    k, v = oracle.dequant_rows(w.k_rows, kt), oracle.dequant_rows(w.v_rows, vt)
    for keys, step in ((k, 0.0 if kt == F16 else 2.0 ** -11), (k.astype(np.float16).astype(np.float64), 0.0)):
        want = attend64(w, keys, v, w.q.astype(np.float64))
        b, bl = bounds(w, keys, v, w.q, want, step)
        assert (np.abs(out - want[0]) <= b).all(), (step, np.max(np.abs(out - want[0]) / b))
        assert (np.abs(lse - want[1]) <= bl).all(), (step, np.abs(lse - want[1]).max() / bl)


def test_the_rounding_of_a_key():
    """The worst product of a scale and a quant lies 2^-11 (and not 2^-12) of itself from
    binary16; with all values of a key so, a logit does.  Sequences of one key: lse is the logit."""
    d = (np.arange(1024, 2048) / 1024.0)[:, None] * np.arange(1.0, 128.0)[None, :]
    e = (d.astype(np.float16).astype(np.float64) - d) / d
    i, j = np.unravel_index(np.argmax(np.abs(e)), e.shape)
    assert 2.0 ** -12 * 1.9 < abs(e[i, j]) <= 2.0 ** -11
    row = np.zeros((2, 4, 8, 34), np.uint8)
    row[..., :2] = np.array([(1024 + i) / 1024.0], np.float16).view(np.uint8)
    row[..., 2:] = j + 1
    w = W.Workload("one", np.array([1, 1], np.int32), 1, 16, 2, Q8, Q8, np.array([[0], [1]], np.int32), row.reshape(2, 4, 272), row.reshape(2, 4, 272),
                   np.ones((2, 1, 24, 256), np.float32), 1 / 16)
    _, lse = decode(w, np.array([2], np.uint32), np.array([0], np.int32), to_dev(w.q).half())
    logit = 16.0 * d[i, j]
    off = np.abs(lse.double().cpu().numpy() - logit)
    assert (off <= (2.0 ** -11 + 2.0 ** -18) * logit).all() and (off > 2.0 ** -12 * 1.9 * logit).all()


def test_values_past_binary16_are_seen():
    """A stored V value past 65504 is infinite: the rows that see it are not finite in
    that dim, whatever its weight, and no other element changes."""
    w, gs, pl = prefix_workload([(2, 700), (1, 500)], [100, 40, 300], 16, Q8, Q8)
    q = to_dev(w.q).half()
    want, want_lse = decode(w, gs, pl, q)
    v = w.v_rows.copy().reshape(len(w.v_rows), 4, 8, 34)
    at = int(w.seq_lens[:1].sum()) + 720  # the second sequence's own row
    v[at, 1, 3, :2] = np.array([3000.0], np.float16).view(np.uint8)
    quants = v[at, 1, 3, 2:].view(np.int8).astype(np.int32)
    bad = W.Workload(w.name, w.seq_lens, 1, 16, w.n_blocks, Q8, Q8, w.table, w.k_rows, v.reshape(w.v_rows.shape), w.q, w.scale)
    out, lse = decode(bad, gs, pl, q)
    past = np.zeros((3, 1, 24, 256), bool)
    past[1, 0, 6:12, 96:128] = np.abs(3000 * quants) > 65504
    block = np.zeros_like(past)
    block[1, 0, 6:12, 96:128] = True
    got = out.cpu().numpy()
    assert past.sum() > 60 and not np.isfinite(got[past]).any() and np.isfinite(got[~past]).all()
    assert np.array_equal(got[~block], want.cpu().numpy()[~block]) and torch.equal(lse, want_lse)
