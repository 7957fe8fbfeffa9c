"""Refusals of the norm + rotation, rotating append, read and shared-prefix
calls: every one returns before any CUDA call (no GPU needed)."""
import ctypes as C

import numpy as np
import pytest

import paged_kv_gqa_11_gb300 as pa
from paged_kv_gqa_11_gb300 import _build

A = 8192  # an aligned address that no call may reach
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load()


def desc(rot=64, inter=0, eps=1e-6, offset=0.0, factor=1.0, freq=0.5):
    return pa.RopeDesc(rot, inter, eps, offset, factor, (C.c_double * 128)(*[freq] * 128))


def norm(lib, d, **kw):
    a = dict(q=A, qs=24 * 256, hq=24, k=A * 2, ks=4 * 256, hk=4, it=1, wq=A, wk=A, wt=1, pos=A, n=1, qo=A * 3, qos=24 * 256, ko=A * 4,
             kos=4 * 256, ot=1)
    a.update(kw)
    return lib.pa_norm_rope(C.addressof(d) if d is not None else None, a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["hk"], a["it"], a["wq"],
                            a["wk"], a["wt"], a["pos"], a["n"], a["qo"], a["qos"], a["ko"], a["kos"], a["ot"], None)


def test_norm_rope_refusals(lib):
    d = desc()
    assert norm(lib, d, n=0) == pa.PA_OK
    inv, uns = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED
    assert norm(lib, None) == inv
    for bad, want in ((dict(rot=24), uns), (dict(rot=272), uns), (dict(inter=2), inv), (dict(eps=-1.0), inv), (dict(eps=float("nan")), inv),
                      (dict(factor=float("inf")), inv), (dict(offset=float("nan")), inv), (dict(freq=float("inf")), inv)):
        assert norm(lib, desc(**bad)) == want, bad
    for kw in (dict(it=2), dict(ot=8), dict(wt=3)):
        assert norm(lib, d, **kw) == uns, kw
    for kw in (dict(q=None), dict(q=A + 8), dict(qo=None), dict(qo=A * 3 + 4), dict(wq=A + 4), dict(pos=None), dict(qs=24 * 256 - 8),
               dict(qs=24 * 256 + 4), dict(hq=0), dict(hq=4097, qs=BIG, qos=BIG), dict(k=None), dict(hk=0), dict(ks=-1024),
               dict(qo=A, ot=0), dict(qo=A, qos=25 * 256), dict(hq=0, q=None, qo=None, hk=0, k=None, ko=None)):
        assert norm(lib, d, **kw) == inv, kw


def append(lib, pool, d, **kw):
    a = dict(kp=A, vp=A, k=A, ks=1024, v=A, vs=1024, it=30, wk=A, wt=30, q=A * 2, qs=24 * 256, hq=24, wq=A, qo=A * 3, qos=24 * 256, qt=30,
             seq=A, pos=A, n=1, tab=A, stride=4, ns=1, err=A)
    a.update(kw)
    return lib.pa_append_rows_rope(pool.handle, a["kp"], a["vp"], C.addressof(d), a["k"], a["ks"], a["v"], a["vs"], a["it"], a["wk"], a["wt"],
                                   a["q"], a["qs"], a["hq"], a["wq"], a["qo"], a["qos"], a["qt"], a["seq"], a["pos"], a["n"], a["tab"],
                                   a["stride"], a["ns"], a["err"], None)


def test_append_rope_refusals(lib):
    pool, d = pa.Pool(8, 16, 4, 256, pa.PA_Q8_0), desc()
    assert append(lib, pool, d, n=0) == pa.PA_OK
    for kw in (dict(kp=None), dict(vp=A + 8), dict(k=None), dict(v=A + 2), dict(ks=1000), dict(vs=1028), dict(seq=None), dict(pos=None),
               dict(tab=None), dict(stride=0), dict(ns=0), dict(err=None), dict(q=None), dict(hq=0), dict(wk=A + 8), dict(qo=A * 2, qt=0)):
        assert append(lib, pool, d, **kw) == pa.PA_ERR_INVALID, kw
    for kw in (dict(it=2), dict(wt=7), dict(qt=2)):
        assert append(lib, pool, d, **kw) == pa.PA_ERR_UNSUPPORTED, kw
    assert append(lib, pool, desc(rot=8)) == pa.PA_ERR_UNSUPPORTED


def test_read_refusals(lib):
    pool = pa.Pool(8, 16, 4, 256, pa.PA_Q4_0)

    def read(kp=A, vp=A, seq=A, pos=A, n=1, tab=A, stride=4, ns=1, ko=A, vo=A, t=1, err=A):
        return lib.pa_read_rows(pool.handle, kp, vp, seq, pos, n, tab, stride, ns, ko, vo, t, err, None)

    assert read(n=0) == pa.PA_OK
    assert read(t=2) == pa.PA_ERR_UNSUPPORTED
    for kw in (dict(ko=None, vo=None), dict(kp=None), dict(vp=None), dict(ko=A + 8), dict(seq=None), dict(pos=None), dict(tab=None),
               dict(stride=0), dict(ns=0), dict(err=None)):
        assert read(**kw) == pa.PA_ERR_INVALID, kw


def test_prefix_refusals(lib):
    pool = pa.Pool(64, 16, 4, 256, pa.PA_Q8_0)

    def call(lens=(40, 50, 30), sizes=(2, 1), pre=(16, 0), t=1, hq=24, q=A, qt=1, out=A, ot=1, ws=A, wsn=BIG, scale=0.0625, stride=4, n=None, err=A,
             sl=True, tab=A):
        sl_, gs, pl = np.array(lens, np.int32), np.array(sizes, np.uint32), np.array(pre, np.int32)
        return pa.pa_decode_prefix(pool, q, qt, A, A, tab, stride, A, sl_ if sl else None, len(lens) if n is None else n, gs, pl, len(sizes), t, hq,
                                   scale, out, ot, None, ws, wsn, err, stream=0, check=False)

    inv, uns = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED
    assert call(lens=(), sizes=(), pre=(), n=0) == pa.PA_OK
    for kw in (dict(t=0), dict(t=97), dict(hq=16), dict(qt=2), dict(ot=8)):
        assert call(**kw) == uns, kw
    for kw in (dict(sizes=(2, 2)), dict(sizes=(1, 1)), dict(sizes=(3, 0)), dict(sizes=(0, 3)), dict(pre=(-1, 0)),
               dict(pre=(40, 0)),               # the new token is each sequence's own
               dict(t=2, pre=(39, 0)), dict(lens=(40, 65, 30)), dict(lens=(40, 50, 0)), dict(q=None), dict(q=A + 8), dict(out=A + 4),
               dict(ws=None), dict(ws=A + 16), dict(scale=0.0), dict(scale=float("nan")), dict(stride=0), dict(err=None), dict(sl=False),
               dict(tab=None), dict(lens=(), sizes=(1,), pre=(0,), n=0)):
        assert call(**kw) == inv, kw
    assert pa.pa_decode_prefix_workspace_size(pool, 3, 2, 97) == 0
