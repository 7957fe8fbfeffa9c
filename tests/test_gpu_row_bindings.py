"""The binding functions over the C calls (addresses, sizes, strides given one by one)
make the calls that the classes make."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_11_gb300 as pa
import workloads as W
from gpu_helpers import device_cache, to_dev
from paged_kv_gqa_11_gb300.cache import PagedKVCache
from paged_kv_gqa_11_gb300.rope import Rope
from rope_helpers import inv_freq, prefix_workload

pytestmark = pytest.mark.gpu
Q8, Q4 = W.TYPE_Q8_0, W.TYPE_Q4_0


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_rows_by_the_binding_and_by_the_classes(dtype):
    """Norm + rotation of parts of a projection with a padded row, the append, the rows
    read back: every argument different from the others, where it can be."""
    rng = np.random.default_rng(7)
    n, hq, hk = 13, 24, 4
    x = torch.from_numpy(rng.standard_normal((n, 33, 256)).astype(np.float32)).cuda().to(dtype)
    q, k, v = x[:, :24], x[:, 24:28], x[:, 28:32]
    wq, wk = (torch.from_numpy((1 + 0.2 * rng.standard_normal(256)).astype(np.float32)).cuda().half() for _ in range(2))
    pos, seq = to_dev(rng.permutation(n).astype(np.int32)), torch.zeros(n, dtype=torch.int32, device="cuda")
    tab = to_dev(np.array([[3, 1]], np.int32))
    r, t = Rope(inv_freq(96), weight_offset=0.5), pa.dtype_number(dtype)
    want = r.apply(q, k, pos, wq, wk, out_dtype=torch.float32)
    qo, ko = torch.empty(n, 30, 256, device="cuda"), torch.empty(n, 7, 256, device="cuda")
    pa.pa_norm_rope(r.address, q, x.stride(0), hq, k, x.stride(0), hk, t, wq, wk, pa.PA_DT_F16, pos, n, qo, qo.stride(0), ko, ko.stride(0), pa.PA_DT_F32)
    assert torch.equal(qo[:, :24], want[0]) and torch.equal(ko[:, :4], want[1])
    a, b = PagedKVCache(5, 16, Q8, Q4), PagedKVCache(5, 16, Q8, Q4)
    want = a.append_rope(r, k, v, seq, pos, tab, k_weight=wk, q=q, q_weight=wq, q_dtype=torch.float16)
    got = torch.empty(n, 25, 256, dtype=torch.float16, device="cuda")
    pa.pa_append_rows_rope(b.pool, b.k_pool, b.v_pool, r.address, k, x.stride(0), v, x.stride(0), t, wk, pa.PA_DT_F16, q, x.stride(0), hq, wq, got,
                           got.stride(0), pa.PA_DT_F16, seq, pos, n, tab, 2, 1, b.err)
    assert torch.equal(got[:, :24], want) and torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)
    # no queries
    c = PagedKVCache(5, 16, Q8, Q4)
    pa.pa_append_rows_rope(c.pool, c.k_pool, c.v_pool, r.address, k, x.stride(0), v, x.stride(0), t, wk, pa.PA_DT_F16, None, 0, 0, None, None, 0,
                           pa.PA_DT_F16, seq, pos, n, tab, 2, 1, c.err)
    assert torch.equal(a.k_pool, c.k_pool) and torch.equal(a.v_pool, c.v_pool)
    want = a.read_rows(seq, pos, tab, dtype=dtype)
    kr, vr = torch.empty(n, 4, 256, dtype=dtype, device="cuda"), torch.empty(n, 4, 256, dtype=dtype, device="cuda")
    pa.pa_read_rows(b.pool, b.k_pool, b.v_pool, seq, pos, n, tab, 2, 1, kr, vr, t, b.err)
    assert torch.equal(kr, want[0]) and torch.equal(vr, want[1])
    for cache in (a, b, c):
        assert cache.check() == pa.PA_OK
    # refusals come as PaError
    for call in (lambda: pa.pa_norm_rope(r.address, q, 1, hq, k, x.stride(0), hk, t, wq, wk, pa.PA_DT_F16, pos, n, qo, qo.stride(0), ko, ko.stride(0),
                                         pa.PA_DT_F32),
                 lambda: pa.pa_append_rows_rope(b.pool, None, b.v_pool, r.address, k, x.stride(0), v, x.stride(0), t, wk, pa.PA_DT_F16, None, 0, 0, None,
                                                None, 0, pa.PA_DT_F16, seq, pos, n, tab, 2, 1, b.err),
                 lambda: pa.pa_read_rows(b.pool, b.k_pool, b.v_pool, seq, pos, n, tab, 2, 1, None, None, t, b.err)):
        with pytest.raises(pa.PaError) as e:
            call()
        assert e.value.status == pa.PA_ERR_INVALID
    with pytest.raises(pa.PaError) as e:
        pa.dtype_number(torch.int8)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED


def test_shared_prefix_by_the_binding_and_by_the_class():
    w, gs, pl = prefix_workload([(3, 500), (1, 20)], [40, 3, 200, 60], 16, Q8, Q4, n_qtok=2)
    cache, tab = device_cache(w)
    q, sl = to_dev(w.q).half(), to_dev(w.seq_lens)
    want, want_lse = cache.decode_prefix(q, tab, sl, w.seq_lens, gs, pl, 2, w.scale, out=torch.empty(q.shape, device="cuda"))
    need = pa.pa_decode_prefix_workspace_size(cache.pool, 4, 2, 2, torch.cuda.current_device())
    out, lse, ws = torch.empty(q.shape, device="cuda"), torch.empty(4, 2, 24, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        out.fill_(7), lse.fill_(7)
        torch.cuda.synchronize()
        rc = pa.pa_decode_prefix(cache.pool, q, pa.PA_DT_F16, cache.k_pool, cache.v_pool, tab, tab.shape[1], sl, w.seq_lens, 4, gs, pl, 2, 2, 24, w.scale,
                                 out, pa.PA_DT_F32, lse, ws, need, cache.err, stream=stream)
        torch.cuda.synchronize()
        assert rc == pa.PA_OK and cache.check() == pa.PA_OK
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
