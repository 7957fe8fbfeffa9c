"""The Rope object: its copies own their constants (no GPU needed)."""
import copy
import ctypes as C
import gc
import pickle

import pytest

import paged_kv_gqa_11_gb300 as pa
from paged_kv_gqa_11_gb300 import PaError, RopeDesc, _build
from paged_kv_gqa_11_gb300.rope import Rope


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def constants(address):
    d = RopeDesc.from_address(address)
    return d.rot_dim, d.interleaved, d.eps, d.weight_offset, d.attn_factor, list(d.inv_freq)


@pytest.mark.parametrize("make", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r)), lambda r: copy.deepcopy({"layer": [r]})["layer"][0]])
def test_copies_read_their_own_constants(make):
    a = Rope([0.5, 0.25] * 8, interleaved=True, eps=0.125, weight_offset=1.0, attn_factor=1.5)
    want = constants(a.address)
    assert want[:5] == (32, 1, 0.125, 1.0, 1.5) and a.address == C.addressof(a.desc)
    b = make(a)
    assert b.address == C.addressof(b.desc) and constants(b.address) == want
    del a
    gc.collect()
    trash = [Rope([3.0] * 8) for _ in range(64)]  # takes up what the original left
    assert constants(b.address) == want and b.address == C.addressof(b.desc)
    del trash


def test_a_copy_is_changed_alone():
    a = Rope([0.5] * 8)
    b = copy.deepcopy(a)
    b.desc.eps = 0.5
    assert constants(b.address)[2] == 0.5 and constants(a.address)[2] != 0.5


@pytest.mark.parametrize("rot_dim", [-2, 1, 33, 65, 257, 258])
def test_widths_that_no_pairs_fill_are_refused(rot_dim):
    with pytest.raises(PaError) as e:
        Rope.from_theta(rot_dim, 1e6)
    assert e.value.status == pa.PA_ERR_INVALID
