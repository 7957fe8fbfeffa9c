"""Compaction of the allocator against a model, frequencies for longer contexts, and the
refusals of the windowed attention and of the calls that move rows and blocks: every one
returns before any CUDA call (no GPU needed)."""
import ctypes as C
import math

import numpy as np
import pytest

import paged_kv_gqa_11_gb300 as pa
from paged_kv_gqa_11_gb300 import _build

A = 8192  # an aligned address that no call may reach
INV, UNS = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load()


@pytest.mark.parametrize("seed", range(20))
def test_compaction(lib, seed):
    """Contents follow their handles: blocks with references of their own, holes anywhere, then allocations and releases
    as before."""
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 40))
    pool = pa.Pool(n, 16)
    held = pool.alloc(int(rng.integers(0, n + 1)))
    if held:
        assert pool.release([h for h in held if rng.random() < 0.5]) == pa.PA_OK
    live = [h for h in held if pool.refcount(h)[0] == pa.PA_OK]
    for h in live:
        assert pool.share([h] * int(rng.integers(0, 3))) == pa.PA_OK
    content = {h & 0xffffffff: (h, pool.refcount(h)[1]) for h in live}
    moves = pool.compact()
    src, dst = [a & 0xffffffff for a, _ in moves], [b & 0xffffffff for _, b in moves]
    m = len(live)
    assert src == sorted(i for i in content if i >= m) and dst == sorted(set(range(m)) - set(content))
    now = dict(zip([a for a, _ in moves], [b for _, b in moves]))
    for h in live:
        rc, count = pool.refcount(now.get(h, h))
        assert (rc, count) == (pa.PA_OK, content[h & 0xffffffff][1])
        if h in now:
            assert pool.refcount(h)[0] == pa.PA_ERR_STALE and pool.release([h]) == pa.PA_ERR_STALE
    assert pool.free_count() == n - m and pool.compact() == []
    rest = pool.alloc(n - m)
    assert [h & 0xffffffff for h in rest] == list(range(m, n))
    assert not set(rest) & set(held)
    every = [now.get(h, h) for h in live]
    assert pool.release(rest + [h for h in every for _ in range(pool.refcount(h)[1])]) == pa.PA_OK and pool.free_count() == n


def test_compaction_refuses_too_small_arrays(lib):
    pool = pa.Pool(10, 16)
    held = pool.alloc(10)
    assert pool.release(held[:6]) == pa.PA_OK
    n, old, new = C.c_uint32(0), (C.c_uint64 * 4)(), (C.c_uint64 * 4)()
    assert lib.pa_compact_blocks(pool.handle, 3, old, new, C.byref(n)) == INV and n.value == 4
    assert all(pool.refcount(h) == (pa.PA_OK, 1) for h in held[6:])  # unchanged
    assert lib.pa_compact_blocks(pool.handle, 4, None, new, C.byref(n)) == INV
    assert lib.pa_compact_blocks(pool.handle, 4, old, new, None) == INV
    assert lib.pa_compact_blocks(None, 4, old, new, C.byref(n)) == INV
    assert lib.pa_compact_blocks(pool.handle, 4, old, new, C.byref(n)) == pa.PA_OK
    assert list(old) == held[6:] and [h & 0xffffffff for h in new] == [0, 1, 2, 3]


def test_frequencies_for_longer_contexts():
    pytest.importorskip("torch")
    from paged_kv_gqa_11_gb300.rope import Rope
    plain = np.array(Rope.from_theta(64, 1e6).desc.inv_freq[:32])
    linear = Rope.scaled(64, 1e6, 4.0, "linear")
    assert np.allclose(linear.desc.inv_freq[:32], plain / 4, rtol=1e-15) and linear.desc.attn_factor == 1.0
    base = np.array(Rope.scaled(64, 1e6, 4.0).desc.inv_freq[:32])
    assert base[0] == 1.0 and math.isclose(base[31], plain[31] / 4, rel_tol=1e-12) and (np.diff(base / plain) < 0).all()
    r = Rope.scaled(64, 1e6, 8.0, "ramp", length=4096)
    f, turns = np.array(r.desc.inv_freq[:32]), 4096 * plain / (2 * np.pi)
    assert (f[turns >= 32] == plain[turns >= 32]).all() and np.allclose(f[turns <= 1], plain[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    k = (turns[mid] - 1) / 31
    assert mid.any() and np.allclose(f[mid], plain[mid] * (k + (1 - k) / 8), rtol=1e-12)
    assert math.isclose(r.desc.attn_factor, 0.1 * math.log(8) + 1, rel_tol=1e-6)
    assert Rope.scaled(64, 1e6, 8.0, "ramp", length=4096, attn_factor=1.0).desc.attn_factor == 1.0
    assert np.allclose(Rope.scaled(64, 1e6, 1.0, "ramp", length=4096).desc.inv_freq[:32], plain, rtol=1e-12)
    for bad in (dict(factor=0.5), dict(factor=float("nan")), dict(factor=2.0, method="other"), dict(factor=2.0, method="ramp"),
                dict(factor=2.0, method="ramp", length=100, fast=1.0), dict(factor=2.0, rot_dim=3), dict(factor=2.0, rot_dim=2)):
        with pytest.raises(pa.PaError):
            Rope.scaled(**{**dict(rot_dim=64, theta=1e6), **bad})


def desc(rot=64, inter=0, eps=1e-6, offset=0.0, factor=1.0, freq=0.5):
    return pa.RopeDesc(rot, inter, eps, offset, factor, (C.c_double * 128)(*[freq] * 128))


def move(lib, pool, rope=None, was=None, **kw):
    a = dict(kp=A, vp=A, ss=A, sp=A, ds=A, dp=A, n=1, st=A, sst=4, sn=1, dt=A, dst=4, dn=1, disjoint=1, ws=None, wb=0, err=A)
    a.update(kw)
    at = lambda d: C.addressof(d) if d is not None else None  # noqa: E731
    return lib.pa_move_rows(pool.handle if pool else None, a["kp"], a["vp"], at(rope), at(was), a["ss"], a["sp"], a["ds"], a["dp"], a["n"],
                            a["st"], a["sst"], a["sn"], a["dt"], a["dst"], a["dn"], a["disjoint"], a["ws"], a["wb"], a["err"], None)


def test_move_rows_refusals(lib):
    pool = pa.Pool(8, 16, 4, 256, pa.PA_Q8_0)
    assert move(lib, pool, n=0) == pa.PA_OK and move(lib, pool, desc(), desc(), n=0) == pa.PA_OK
    assert move(lib, None) == INV
    for kw in (dict(kp=None), dict(vp=None), dict(kp=A + 8), dict(vp=A + 4), dict(ss=None), dict(sp=None), dict(ds=None), dict(dp=None),
               dict(st=None), dict(dt=None), dict(sst=0), dict(dst=0), dict(sn=0), dict(dn=0), dict(sst=1 << 31), dict(dn=1 << 31),
               dict(err=None)):
        assert move(lib, pool, **kw) == INV, kw
    for bad, want in ((dict(rot=24), UNS), (dict(rot=272), UNS), (dict(inter=2), INV), (dict(factor=float("inf")), INV),
                      (dict(freq=float("nan")), INV)):
        assert move(lib, pool, desc(**bad)) == want, bad
        assert move(lib, pool, desc(), desc(**bad)) == want, bad
    assert move(lib, pool, None, desc()) == INV
    assert move(lib, pool, desc(64), desc(32)) == INV and move(lib, pool, desc(), desc(inter=1)) == INV
    assert move(lib, pool, desc(), desc(factor=0.0)) == INV and move(lib, pool, desc(factor=0.0)) == INV
    need = lib.pa_move_rows_workspace_size(pool.handle, 1000)
    assert need == 1000 * 4 * 2 * 272 and lib.pa_move_rows_workspace_size(pool.handle, 64) == 0 < lib.pa_move_rows_workspace_size(pool.handle, 65)
    for kw in (dict(ws=None, wb=need), dict(ws=A, wb=need - 1), dict(ws=A + 8, wb=need)):
        assert move(lib, pool, disjoint=0, n=1000, **kw) == INV, kw


def test_move_blocks_refusals(lib):
    pool = pa.Pool(8, 16, 4, 256, pa.PA_Q8_0)
    call = lambda kp=A, vp=A, src=A, dst=A, n=1, t=A, o=A, e=4, err=A: lib.pa_move_blocks(pool.handle, kp, vp, src, dst, n, t, o, e, err, None)  # noqa: E731
    assert call(n=0, e=0) == pa.PA_OK
    for kw in (dict(kp=None), dict(vp=None), dict(kp=A + 8), dict(src=None), dict(dst=None), dict(t=None), dict(o=None), dict(err=None)):
        assert call(**kw) == INV, kw
    assert call(e=1 << 41) == UNS and call(n=1 << 31) == UNS


def attend(lib, pool, lens=(100, 50), new=(3, 1), **kw):
    a = dict(q=A, qs=24 * 256, qt=1, kp=A, vp=A, tab=A, stride=8, dev=A, ns=len(lens or new), hq=24, window=0, sinks=0, scale=0.0625, out=A,
             os=24 * 256, ot=1, lse=A, ws=A, wb=0, err=A)
    a.update(kw)
    arr = lambda x: None if x is None else (C.c_int32 * max(1, len(x)))(*x)  # noqa: E731
    return lib.pa_attend_window(pool.handle, a["q"], a["qs"], a["qt"], a["kp"], a["vp"], a["tab"], a["stride"], a["dev"], arr(lens), arr(new),
                                a["ns"], a["hq"], a["window"], a["sinks"], a["scale"], a["out"], a["os"], a["ot"], a["lse"], a["ws"], a["wb"],
                                a["err"], None)


def test_attend_window_refusals(lib):
    pool = pa.Pool(64, 16, 4, 256, pa.PA_Q8_0)
    assert attend(lib, pool, ns=0) == pa.PA_OK and attend(lib, pool, new=(0, 0)) == pa.PA_OK
    for kw in (dict(hq=20), dict(hq=0), dict(qt=2), dict(ot=8)):
        assert attend(lib, pool, **kw) == UNS, kw
    for kw in (dict(lens=None, ns=2), dict(new=None), dict(new=(3, -1)), dict(new=(3, 51)), dict(lens=(100, 129)), dict(lens=(-5, 50)),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(q=None), dict(out=None),
               dict(kp=None), dict(vp=None), dict(tab=None), dict(dev=None), dict(ws=None), dict(err=None), dict(q=A + 8), dict(out=A + 4),
               dict(kp=A + 8), dict(vp=A + 8), dict(ws=A + 128), dict(qs=24 * 256 - 8), dict(qs=24 * 256 + 4), dict(os=-1), dict(stride=0),
               dict(os=(1 << 40) + 8)):
        assert attend(lib, pool, **{**dict(lens=(100, 50)), **kw}) == INV, kw
    big = pa.Pool(4, 1 << 20, 4, 256, pa.PA_Q8_0)
    assert attend(lib, big, lens=(1 << 25,), new=(1 << 25,), stride=1 << 10) == UNS  # new tokens
    assert attend(lib, big, lens=(0x7fffffff,), new=(1,), stride=1 << 12) == UNS  # past what a tile can count
    wide = pa.Pool(1, 16, 4096, 256, pa.PA_Q8_0)
    assert attend(lib, wide, lens=(1 << 26,), new=(1,), stride=1 << 22, hq=6 * 4096, qs=6 << 20, os=6 << 20) == UNS  # tiles of a launch
