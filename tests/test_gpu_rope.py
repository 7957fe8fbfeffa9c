"""Norm + rotation, the rotating append and cache reads against float64.

Tolerance of the norm and rotation, counted in half steps of fp32 (u = 2^-24):
the sum of 256 squares is 8 fused steps in a lane and 5 shuffle sums, 13 u, of
which the square root takes half; the mean and eps 2 u / 2; the reciprocal square
root 2 units in the last place, 4 u; the weight with its offset 1 u; two products
2 u -- under 15 u of each value of the pair.  Cosine and sine: the phase as a
float, 2^-25 half-turns, is pi * 2^-25 < 2 u in the angle, its truncation to 32
bits 2^-32 turns < 1 u, sincospi 2 units in the last place at most 4 u, the factor
1 u; the product and sum of the rotation 2 u.  Together under 25 u (|a| + |b|),
plus half a step of the output's type."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import to_dev
from paged_kv_gqa_11_gb300 import PA_ERR_BOUNDS, PA_OK, PaError
from paged_kv_gqa_11_gb300.cache import PagedKVCache
from paged_kv_gqa_11_gb300.rope import Rope
from rope_helpers import inv_freq, norm_rope64

pytestmark = pytest.mark.gpu
F16, Q4, Q8 = W.TYPE_F16, W.TYPE_Q4_0, W.TYPE_Q8_0
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def bound(want, mag, dtype, factor=1.0):
    half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]
    tiny = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[dtype]
    e = 25 * U * mag * max(1.0, abs(factor))
    return e + half * (np.abs(want) + e) + tiny


def check(got, want, mag, factor=1.0, what=""):
    err = np.abs(got.double().cpu().numpy() - want)
    b = bound(want, mag, got.dtype, factor)
    assert np.isfinite(err).all() and (err <= b).all(), f"{what}: {np.max(err / b):.3g} of the bound"


def rows(rng, n, h, dtype, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal((n, h, 256))).astype(np.float32)).cuda().to(dtype)


@pytest.mark.parametrize("n,hq,hk,i,o,wt,rot,inter", [
    (1, 24, 4, "bf16", "bf16", "bf16", 64, False),
    (7, 24, 4, "f16", "f32", "f32", 256, False),
    (33, 24, 4, "f32", "f16", "f16", 128, True),
    (5, 1, 3, "bf16", "f32", "f32", 16, False),
    (3, 2, 1, "f32", "f32", "bf16", 96, False),
    (700, 24, 4, "bf16", "f16", "bf16", 256, True),
    (4, 3, 1, "f16", "bf16", "f16", 0, False),
    (2000, 6, 2, "f32", "f32", "f32", 32, True),
])
def test_norm_rope(n, hq, hk, i, o, wt, rot, inter):
    rng = np.random.default_rng(n + rot)
    q, k = rows(rng, n, hq, DT[i], 3.0), rows(rng, n, hk, DT[i], 0.2)
    wq, wk = (torch.from_numpy((1 + 0.3 * rng.standard_normal(256)).astype(np.float32)).cuda().to(DT[wt]) for _ in range(2))
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    freq = inv_freq(rot) if rot else []
    r = Rope(freq, interleaved=inter)
    qo, ko = r.apply(q, k, to_dev(pos), wq, wk, out_dtype=DT[o])
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        want, mag = norm_rope64(x.double().cpu().numpy(), pos, freq, inter, w.double().cpu().numpy())
        check(y, want, mag, what=f"{n} {i}->{o}")


def test_norm_rope_positions_and_constants():
    """The ends of int32, zero, negative positions; a factor, a weight offset, a
    large eps; fast frequencies (more than a turn a position)."""
    rng = np.random.default_rng(3)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131072, 1 << 24], np.int32)
    freq = [2.0 ** (7 - i) if i < 16 else 10000.0 ** (-i / 64) for i in range(64)]
    x = rows(rng, len(pos), 5, torch.float32)
    w = torch.from_numpy((0.3 * rng.standard_normal(256)).astype(np.float32)).cuda()
    y, _ = Rope(freq, eps=0.25, weight_offset=1.0, attn_factor=1.25).apply(x, None, to_dev(pos), w)
    # the float64 angle itself is off by 2^-53 of up to 2^38 radians: keep to |p f| < 2^24 there
    ok = np.abs(pos.astype(np.float64)) * max(freq) < 2.0 ** 24
    want, mag = norm_rope64(x.cpu().numpy(), pos, freq, False, w.cpu().numpy(), 0.25, 1.0, 1.25)
    check(y[torch.from_numpy(ok).cuda()], want[ok], mag[ok], 1.25)
    slow = [f for f in freq if f < 1] + [0.001] * 16
    y, _ = Rope(slow).apply(x, None, to_dev(pos))  # no weight: only rotated
    want, mag = norm_rope64(x.cpu().numpy(), pos, slow)
    # here 2^31 radians at most, off by 2^-22 in float64: angles in integers instead
    from fractions import Fraction
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    ang = np.array([[float((Fraction(int(p)) * Fraction(f)) % two_pi) for f in slow] for p in pos])
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    h = len(slow)
    x64 = x.double().cpu().numpy()
    a, b = x64[..., :h], x64[..., h:2 * h]
    want[..., :h], want[..., h:2 * h] = a * c - b * s, b * c + a * s
    check(y, want, mag)


def test_norm_rope_zero_rows_and_zero_heads_of_values():
    r = Rope(inv_freq(64))
    z = torch.zeros(3, 2, 256, device="cuda")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    y, _ = r.apply(z, None, pos, torch.ones(256, device="cuda"))
    assert torch.equal(y, z)
    e = torch.empty(0, 2, 256, device="cuda")
    y, _ = r.apply(e, None, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert y.shape == e.shape


@pytest.mark.parametrize("rot,inter", [(64, False), (256, False), (128, True)])
def test_norm_rope_in_place_and_strided(rot, inter):
    """Parts of one projection with a padded row, in place and out of place, equal
    bit for bit; the rest of the projection stays."""
    rng = np.random.default_rng(rot)
    n = 37
    base = rows(rng, n, 33, torch.bfloat16)
    pos = to_dev(rng.integers(0, 5000, n).astype(np.int32))
    w = torch.rand(256, device="cuda").to(torch.bfloat16)
    r = Rope(inv_freq(rot), interleaved=inter)
    a, b = r.apply(base[:, :24].contiguous(), base[:, 24:28].contiguous(), pos, w, w)
    keep = base.clone()
    r.apply(base[:, :24], base[:, 24:28], pos, w, w, q_out=base[:, :24], k_out=base[:, 24:28])
    assert torch.equal(base[:, :24], a) and torch.equal(base[:, 24:28], b) and torch.equal(base[:, 28:], keep[:, 28:])


# ------------------------------------------------------------------ append

def places(rng, lens, ps, start=0):
    seq = np.repeat(np.arange(len(lens)), lens).astype(np.int32)
    pos = np.concatenate([start + np.arange(n) for n in lens]).astype(np.int32)
    pages = -(-(start + max(lens)) // ps)
    order = rng.permutation(len(lens) * pages + 3).astype(np.int32)
    return seq, pos, order[:len(lens) * pages].reshape(len(lens), pages), len(lens) * pages + 3


@pytest.mark.parametrize("kt,vt,ps,lens", [(F16, Q4, 16, [40, 3]), (Q8, Q8, 48, [1]), (Q4, F16, 256, [300, 16, 17])])
def test_append_without_rotation_equals_plain_append(kt, vt, ps, lens):
    """No weight, no rotation: byte for byte what pa_append_rows_f16 stores, edge
    blocks included (zero blocks, ties in magnitude, tiny scales)."""
    rng = np.random.default_rng(1)
    seq, pos, table, nb = places(rng, lens, ps)
    n = len(seq)
    x = rng.standard_normal((2, n, 4, 256)).astype(np.float16)
    x[0, 0, 0, :32] = 0
    x[0, 0, 1, :32] = np.linspace(-2, 2, 32)
    x[1, 0, 2, 32:64] = np.linspace(2, -2, 32)
    x[1, 0, 3, :32] *= np.float16(1e-5)
    k, v = to_dev(x[0]), to_dev(x[1])
    a, b = PagedKVCache(nb, ps, kt, vt), PagedKVCache(nb, ps, kt, vt)
    tab, s, p = to_dev(table), to_dev(seq), to_dev(pos)
    a.append_f16(k, v, s, p, tab)
    for dt in (torch.float16, torch.float32):
        b.k_pool.zero_(), b.v_pool.zero_()
        b.append_rope(Rope([]), k.to(dt), v.to(dt), s, p, tab)
        assert b.check() == PA_OK
        assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)


def stored_bound(x, t, err):
    """Half a quantisation step of each 32-block (a Q4_0 value past 7 steps is cut to 7), the scale's rounding to
    binary16, and the value's own error."""
    if t == F16:
        return 2.0 ** -11 * (np.abs(x) + err) + 2.0 ** -25 + err
    b = np.abs(x).reshape(*x.shape[:-1], 8, 32)
    top = b.max(-1, keepdims=True) + err.reshape(b.shape).max(-1, keepdims=True)
    step = top / (127 if t == Q8 else 8)
    # the rule's own roundings in fp32 move a value by less than 1e-5 steps
    e = step * (0.5 + 1e-4) if t == Q8 else np.where(b > 7.4 * step, step * 1.0001, step * (0.5 + 1e-4))
    return (e + 2.0 ** -11 * (b + step) + 2.0 ** -25 * 128).reshape(x.shape) + err


@pytest.mark.parametrize("kt,vt,ps,lens,start,i,rot,inter", [
    (Q8, Q4, 16, [5], 1000, "bf16", 64, False),
    (Q4, Q8, 48, [90, 33, 1], 0, "f16", 256, False),
    (F16, F16, 256, [300, 20], 70000, "f32", 128, True),
    (Q8, Q8, 32, [2500], 5, "bf16", 256, False),
])
def test_append_rope(kt, vt, ps, lens, start, i, rot, inter):
    """A fused projection: keys normalised, rotated and stored, values stored,
    queries returned; the stored rows read back; other rows stay as they were."""
    rng = np.random.default_rng(rot + len(lens))
    seq, pos, table, nb = places(rng, lens, ps, start)
    n = len(seq)
    qkv = rows(rng, n, 32, DT[i], 2.0)
    wq, wk = (torch.from_numpy((1 + 0.3 * rng.standard_normal(256)).astype(np.float32)).cuda().to(DT[i]) for _ in range(2))
    c = PagedKVCache(nb, ps, kt, vt)
    c.k_pool.fill_(0x5a), c.v_pool.fill_(0x5a)
    r = Rope(inv_freq(rot), interleaved=inter)
    tab, s, p = to_dev(table), to_dev(seq), to_dev(pos)
    q = c.append_rope(r, qkv[:, 24:28], qkv[:, 28:], s, p, tab, k_weight=wk, q=qkv[:, :24], q_weight=wq)
    k, v = c.read_rows(s, p, tab, dtype=torch.float32)
    assert c.check() == PA_OK
    x = qkv.double().cpu().numpy()
    want, mag = norm_rope64(x[:, :24], pos, inv_freq(rot), inter, wq.double().cpu().numpy())
    check(q, want, mag, what="q")
    want, mag = norm_rope64(x[:, 24:28], pos, inv_freq(rot), inter, wk.double().cpu().numpy())
    e = np.abs(k.double().cpu().numpy() - want)
    assert (e <= stored_bound(want, kt, 25 * U * mag)).all()
    e = np.abs(v.double().cpu().numpy() - x[:, 28:])
    assert (e <= stored_bound(x[:, 28:], vt, np.zeros_like(e))).all()
    # bytes of rows that no row of the call owns
    for pool, t, role in ((c.k_pool, kt, oracle.ROLE_K), (c.v_pool, vt, oracle.ROLE_V)):
        mark = np.zeros(pool.numel(), np.uint8)
        oracle.scatter(mark, nb, 4, ps, t, role, np.ones((n, 4, oracle.row_bytes(t)), np.uint8), seq, pos, table)
        got = pool.cpu().numpy()
        assert (got[mark == 0] == 0x5a).all()


def test_append_rope_padding_rows():
    """Rows of a padded batch (no sequence, a position or page outside the table,
    a bad table entry) are reported and not stored; their queries come back."""
    rng = np.random.default_rng(8)
    c = PagedKVCache(8, 16, Q8, Q4)
    table = np.array([[0, 1, 99], [2, 3, -1]], np.int32)
    seq = np.array([0, -1, 1, 0, 2, 1], np.int32)
    pos = np.array([5, 6, 40, 48, 0, 17], np.int32)
    x = rows(rng, 6, 32, torch.float16)
    r = Rope(inv_freq(64))
    q = c.append_rope(r, x[:, 24:28], x[:, 28:], to_dev(seq), to_dev(pos), to_dev(table), q=x[:, :24])
    assert c.check() == PA_ERR_BOUNDS
    want, mag = norm_rope64(x[:, :24].double().cpu().numpy(), pos, inv_freq(64))
    check(q, want, mag)
    d = PagedKVCache(8, 16, Q8, Q4)
    good = [0, 5]
    d.append_rope(r, x[good][:, 24:28], x[good][:, 28:], to_dev(seq[good]), to_dev(pos[good]), to_dev(table))
    assert d.check() == PA_OK
    assert torch.equal(c.k_pool, d.k_pool) and torch.equal(c.v_pool, d.v_pool)
    # reading such rows gives zeros and the report
    k, v = c.read_rows(to_dev(seq), to_dev(pos), to_dev(table))
    assert c.check() == PA_ERR_BOUNDS
    bad = [1, 2, 3, 4]
    assert not k[bad].any() and not v[bad].any() and k[good].any() and v[good].any()


@pytest.mark.parametrize("kt,vt", [(F16, Q8), (Q4, F16), (Q8, Q4)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_read_rows_matches_oracle(kt, vt, dtype):
    """Bit for bit: the stored value is exact in fp32, then rounded once."""
    w = W.make_workload("read", 9, [300, 17, 1], 48, kt, vt, 1, "shuffled")
    c = PagedKVCache(w.n_blocks, w.page_size, kt, vt)
    tab = to_dev(w.table)
    c.append(to_dev(w.k_rows), to_dev(w.v_rows), to_dev(w.row_seq), to_dev(w.row_pos), tab)
    pick = np.random.default_rng(2).integers(0, len(w.row_seq), 500)  # any order, repeats
    k, v = c.read_rows(to_dev(w.row_seq[pick]), to_dev(w.row_pos[pick]), tab, dtype=DT[dtype])
    assert c.check() == PA_OK
    for got, src, t in ((k, w.k_rows, kt), (v, w.v_rows, vt)):
        want = torch.from_numpy(oracle.dequant_rows(src[pick], t).astype(np.float32)).to(DT[dtype])
        assert torch.equal(got.cpu(), want.reshape(got.shape))
    only = torch.full_like(v, 7.0)
    c.read_rows(to_dev(w.row_seq[pick]), to_dev(w.row_pos[pick]), tab, v_out=only)
    assert torch.equal(only, v)


def test_rope_step_captured_and_on_another_stream():
    """Append, read and rotate captured once and replayed on new inputs, and the
    same on a side stream, equal the plain calls."""
    rng = np.random.default_rng(4)
    seq, pos, table, nb = places(rng, [9, 4], 16, 100)
    tab, s, p = to_dev(table), to_dev(seq), to_dev(pos)
    r = Rope(inv_freq(64))
    w = torch.rand(256, device="cuda")
    xs = [rows(rng, len(seq), 32, torch.bfloat16) for _ in range(3)]

    def step(c, x, stream=None):
        q = c.append_rope(r, x[:, 24:28], x[:, 28:], s, p, tab, k_weight=w.bfloat16(), q=x[:, :24], stream=stream)
        return (q, *c.read_rows(s, p, tab, stream=stream))

    want = [step(PagedKVCache(nb, 16, Q8, Q8), x) for x in xs]
    c = PagedKVCache(nb, 16, Q8, Q8)
    x = xs[0].clone()
    step(c, x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(c, x)
    for src, ref in zip(xs, want):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(c, xs[1])
    got2 = step(c, xs[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1])) and all(torch.equal(a, b) for a, b in zip(got2, want[1]))


def test_unknown_types_are_refused():
    r = Rope(inv_freq(64))
    with pytest.raises(PaError):
        r.apply(torch.zeros(1, 1, 256, dtype=torch.float64, device="cuda"), None, torch.zeros(1, dtype=torch.int32, device="cuda"))


def test_refusals_of_the_python_calls():
    r = Rope(inv_freq(64))
    dev = "cuda"
    x = torch.zeros(3, 32, 256, dtype=torch.float16, device=dev)
    pos = torch.zeros(3, dtype=torch.int32, device=dev)
    q, k, v = x[:, :24], x[:, 24:28], x[:, 28:]
    for args, kw in [((None, None, pos), {}), ((q.cpu(), None, pos), {}), ((q, k.float(), pos), {}), ((q, k[:2], pos), {}), ((q, k, pos.long()), {}),
                     ((q, k, pos[:2]), {}), ((q, k, pos.cpu()), {}), ((q[0], None, pos), {}), ((q[..., :128], None, pos), {}),
                     ((q[:, ::2], None, pos), {}), ((q[:, :, ::1].transpose(0, 1), None, pos), {}), ((q[:1].expand(3, 24, 256), None, pos), {}),
                     ((q, None, pos), dict(k_out=torch.empty_like(k))), ((q, None, pos), dict(q_out=torch.empty_like(k))),
                     ((q, None, pos), dict(q_out=torch.empty_like(q), out_dtype=torch.float32)), ((q, None, pos), dict(out_dtype=torch.float64)),
                     ((q, None, pos), dict(out_dtype="half")), ((q, None, pos), dict(q_weight=x[0, 0, :128])), ((q, None, pos), dict(q_weight=x[0, 0].double())),
                     ((q, k, pos), dict(q_weight=x[0, 0], k_weight=x[0, 0].float())), ((q, None, pos), dict(stream="s"))]:
        with pytest.raises(PaError):
            r.apply(*args, **kw)
    c = PagedKVCache(8, 16, Q8, Q8)
    seq = torch.zeros(3, dtype=torch.int32, device=dev)
    tab = torch.zeros(1, 4, dtype=torch.int32, device=dev)
    for args, kw in [((k, v[:, :2], seq, pos, tab), {}), ((k, v.float(), seq, pos, tab), {}), ((q, q, seq, pos, tab), {}), ((k, v, seq[:2], pos, tab), {}),
                     ((k, v, seq, pos, tab.long()), {}), ((k, v, seq, pos, tab[0]), {}), ((k, v, seq.cpu(), pos, tab), {}),
                     ((k, v, seq, pos, tab), dict(q_out=torch.empty_like(q))), ((k, v, seq, pos, tab), dict(q=q.float())),
                     ((k, v, seq, pos, tab), dict(q=q, q_out=torch.empty_like(q), q_dtype=torch.float32))]:
        with pytest.raises(PaError):
            c.append_rope(r, *args, **kw)
    for args, kw in [((seq, pos[:2], tab), {}), ((seq[None], pos, tab), {}), ((seq, pos, tab.cpu()), {}), ((seq, pos, tab), dict(dtype=torch.int8)),
                     ((seq, pos, tab), dict(k_out=torch.empty(3, 4, 128, device=dev))), ((seq, pos, tab), dict(k_out=torch.empty(2, 4, 256, device=dev))),
                     ((seq, pos, tab), dict(k_out=torch.empty(3, 4, 256, device=dev), v_out=torch.empty(3, 4, 256, device=dev).half()))]:
        with pytest.raises(PaError):
            c.read_rows(*args, **kw)
    torch.cuda.synchronize()
    assert c.check() == PA_OK and not c.k_pool.any() and not c.v_pool.any()
    # no rows: empty outputs, nothing launched
    none = torch.empty(0, dtype=torch.int32, device=dev)
    assert r.apply(q[:0], k[:0], none)[0].shape == (0, 24, 256) and c.read_rows(none, none, tab)[0].shape == (0, 4, 256)
    assert c.append_rope(r, k[:0], v[:0], none, none, tab, q=q[:0]).shape == (0, 24, 256)
