"""Norm + rotation: values that the rotation does not reach stay what they are."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from paged_kv_gqa_11_gb300.rope import Rope
from rope_helpers import inv_freq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rot,inter", [(0, False), (64, False), (64, True), (240, True), (128, False)])
@pytest.mark.parametrize("weight", [False, True])
def test_values_past_the_rotation_stay(dtype, rot, inter, weight):
    """Without a weight bit for bit (infinities and negative zeros among them, NaN as NaN);
    with one, the value times weight and norm, whatever stands beside it."""
    x = torch.from_numpy(np.random.default_rng(rot).standard_normal((5, 3, 256)).astype(np.float32)).cuda().to(dtype)
    special = [float("inf"), float("-inf"), float("nan"), -0.0, 0.0]
    at = [rot + 1, rot + 4, rot + 9, rot + 11, 255]
    pos = torch.tensor([0, 1, 77, -3, 1 << 20], dtype=torch.int32, device="cuda")
    r = Rope(inv_freq(rot) if rot else [], interleaved=inter)
    if not weight:
        plain, _ = r.apply(x, None, pos)
        y = x.clone()
        for i, v in zip(at, special):
            y[:, :, i] = v
        got, _ = r.apply(y, None, pos)
        past, was = got[..., rot:].contiguous(), y[..., rot:].contiguous()
        assert torch.equal(past.isnan(), was.isnan())
        past[past.isnan()], was[was.isnan()] = 0, 0
        assert torch.equal(past.view(torch.uint8), was.view(torch.uint8))
        assert torch.equal(got[..., :rot], plain[..., :rot])
        return
    # zeros of either sign keep their sign under a positive weight
    w = (torch.rand(256, device="cuda") + 0.5).to(dtype)
    y = x.clone()
    y[:, :, at[3]], y[:, :, at[4]] = -0.0, 0.0
    got, _ = r.apply(y, None, pos, w)
    assert (got[:, :, at[3]].float().signbit() & (got[:, :, at[3]] == 0)).all() and (~got[:, :, at[4]].float().signbit()).all()
    # an infinite value makes the norm infinite: it is NaN itself (inf / inf), the rest zeros
    y[:, :, at[0]] = float("inf")
    got, _ = r.apply(y, None, pos, w)
    assert got[:, :, at[0]].isnan().all()
    rest = [i for i in range(rot, 256) if i != at[0]]
    assert (got[:, :, rest] == 0).all()


def test_infinite_values_in_the_rotated_part_touch_their_pair_only():
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((4, 2, 256)).astype(np.float32)).cuda()
    pos = torch.tensor([3, 5, 9, 1000], dtype=torch.int32, device="cuda")
    for inter, pair in ((False, [10, 42]), (True, [10, 11])):
        r = Rope(inv_freq(64), interleaved=inter)
        plain, _ = r.apply(x, None, pos)
        y = x.clone()
        y[:, :, 10] = float("inf")
        got, _ = r.apply(y, None, pos)
        rest = [i for i in range(256) if i not in pair]
        assert torch.equal(got[:, :, rest], plain[:, :, rest])
        assert not got[:, :, pair].isfinite().any()


@pytest.mark.parametrize("inter", [False, True])
def test_cosines_and_sines(inter):
    """Pairs (1, 0) turn into (cos, sin), exactly: both within 5 u of float64's (u = 2^-24).
    The phase's cut to 32 bits is u / 32 of an angle, its three fp32 roundings 3 u pi / 4, the
    series' remainder u / 2, its evaluation below 1.5 u; float64 itself is off by 2^-30 at
    angles below 2^24."""
    rng = np.random.default_rng(2)
    pos = np.concatenate([np.arange(-64, 64), rng.integers(-(1 << 24), 1 << 24, 8000)]).astype(np.int32)
    freq = [1.0, np.pi / 4, np.pi / 8, 0.5] + [float(x) for x in rng.uniform(0, 1, 60)] + [1e-3 ** (i / 64) for i in range(64)]
    x = torch.zeros(len(pos), 1, 256, device="cuda")
    (x[..., 0::2] if inter else x[..., :128]).fill_(1.0)
    y, _ = Rope(freq, interleaved=inter).apply(x, None, to_dev(pos))
    y = y[:, 0].double().cpu().numpy()
    c, s = (y[:, 0::2], y[:, 1::2]) if inter else (y[:, :128], y[:, 128:])
    ang = pos.astype(np.float64)[:, None] * np.array(freq)
    worst = max(np.abs(c - np.cos(ang)).max(), np.abs(s - np.sin(ang)).max())
    assert worst < 5 * 2.0 ** -24 + 2.0 ** -28, worst * 2 ** 24


def test_a_single_row_of_any_stride():
    """One row of a buffer whose rows are no whole 16 bytes long: its stride is never used."""
    buf = torch.from_numpy(np.random.default_rng(6).standard_normal((8, 28 * 256 + 4)).astype(np.float32)).cuda().half()
    row = buf[:, :28 * 256].unflatten(1, (28, 256))[2:3]
    assert row.stride(0) % 8 and row.data_ptr() % 16 == 0
    pos, w, r = torch.tensor([9], dtype=torch.int32, device="cuda"), torch.rand(256, device="cuda").half(), Rope(inv_freq(64))
    want = r.apply(row[:, :24].contiguous(), row[:, 24:].contiguous(), pos, w, w)
    got = r.apply(row[:, :24], row[:, 24:], pos, w, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    r.apply(row[:, :24], row[:, 24:], pos, w, w, q_out=row[:, :24], k_out=row[:, 24:])
    assert torch.equal(row[:, :24], want[0]) and torch.equal(row[:, 24:], want[1])
