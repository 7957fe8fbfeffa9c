"""Pool buffers that a caller brings to PagedKVCache: refused, before anything is
made on a GPU, where the kernels could not use them."""
import pytest
import torch

import workloads as W
from paged_kv_gqa_11_gb300 import PA_ERR_INVALID, PA_OK, PaError, _build
from paged_kv_gqa_11_gb300.cache import PagedKVCache

Q8, F16 = W.TYPE_Q8_0, W.TYPE_F16
N = 4 * 4 * 16 * 272  # bytes of four Q8_0 blocks of 16 rows


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


@pytest.mark.parametrize("device", ["cuda", "cuda:0"])
def test_host_memory_is_refused(device):
    host = torch.zeros(N, dtype=torch.uint8)
    for kw in (dict(k_pool=host, v_pool=host), dict(k_pool=host)):
        with pytest.raises(PaError) as e:
            PagedKVCache(4, 16, Q8, device=device, **kw)
        assert e.value.status == PA_ERR_INVALID


@pytest.mark.gpu
def test_buffers_that_do_not_fit_are_refused():
    good = torch.zeros(N, dtype=torch.uint8, device="cuda")
    for bad in (good.cpu(), good[:-1], torch.zeros(N + 8, dtype=torch.uint8, device="cuda")[8:], torch.zeros(2 * N, dtype=torch.uint8, device="cuda")[::2],
                good.view(torch.int32), good.float()):
        for kw in (dict(k_pool=bad, v_pool=good), dict(k_pool=good, v_pool=bad), dict(v_pool=bad)):
            with pytest.raises(PaError) as e:
                PagedKVCache(4, 16, Q8, **kw)
            assert e.value.status == PA_ERR_INVALID
    # one of the caller's, one of the cache's own; either way of naming the device
    for device in ("cuda", "cuda:0", torch.device("cuda", 0)):
        c = PagedKVCache(4, 16, Q8, device=device, k_pool=good)
        assert c.k_pool is good and c.v_pool.numel() == N and c.check() == PA_OK
