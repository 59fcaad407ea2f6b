"""Scales of rotated keys whose largest magnitude lies next to a border between two scales: the exact product decides."""
import numpy as np
import pytest
import torch

import near_ties
import paged_ref as ref
from test_gpu_paged import Cache, E4M3, INT8, ok

pytestmark = pytest.mark.gpu

BORDER = {E4M3: 3.5, INT8: 3.96875}                                  # 448 * 2^-7, 127 * 2^-5


def rows_of(w, fmt):
    """The witness pairs as keys: pair i mod 8 of 16 turned dims, half layout at offset 8."""
    x = np.zeros((len(w), 2, 128))
    i = np.arange(len(w))
    x[i, 1, 8 + i % 8], x[i, 1, 16 + i % 8] = w[:, 1], w[:, 2]
    x[i, 0, 100] = 1.0                                               # the other head: never in doubt
    return x


def fp32_scale_differs(w, fmt):
    """How many rows would get another scale from the fp32 rotation."""
    c, s = np.cos(w[:, 0]).astype(np.float32), np.sin(w[:, 0]).astype(np.float32)
    y32 = w[:, 1].astype(np.float32) * c - w[:, 2].astype(np.float32) * s
    y, _ = near_ties.turned(w[:, 0], w[:, 1], w[:, 2])
    return int(((np.abs(y32) > BORDER[fmt]) != (np.abs(y) > BORDER[fmt])).sum())


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("form", ["one token each", "five of few", "five of many"])
def test_scale_next_to_a_border(cuda_ok, fmt, form):
    """Largest magnitudes within 2^-23 of a border, on both sides of it, in calls of one, two and four rows a thread."""
    count = {"one token each": 300, "five of few": 40, "five of many": 700}[form]
    w = near_ties.near([BORDER[fmt], -BORDER[fmt]], 3, count)
    assert fp32_scale_differs(w, fmt) > count // 20
    per = 1 if form == "one token each" else 5
    x = np.zeros((count * per, 2, 128))
    x[per // 2::per] = rows_of(w, fmt)
    pos = np.arange(count * per) % 7
    pos[per // 2::per] = w[:, 0]
    k = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(k.double().numpy(), x)
    cache = Cache([per] * count, 16, 2, fmt)
    cache.append(k.cuda(), k.cuda(), [0] * count, None if per == 1 else [per] * count,
                 inv_freq=torch.ones(8, dtype=torch.float64).cuda(), rot_offset=8,
                 rope_pos=torch.from_numpy(pos.astype(np.int32)).cuda())
    ok()
    got, _, ks, _ = cache.cpu()
    y, _ = near_ties.turned(w[:, 0], w[:, 1], w[:, 2])
    want = np.array([2.0 ** ref.exponent(float(abs(v)) if abs(v) != BORDER[fmt] else 0, fmt) for v in y])
    pid = cache.table[:, 0].long()
    assert np.array_equal(ks[pid, 1].double().numpy(), want)
    assert torch.all(ks[pid, 0] == 2.0 ** ref.exponent(1.0, fmt))
    # and the largest itself is stored as the nearest of its scale
    i = np.arange(count)
    stored = got[pid, per // 2, 1][i, 8 + i % 8].double().numpy()
    assert np.array_equal(stored, ref.round8((y / want).astype(np.float64), fmt))


def test_scale_next_to_a_border_of_a_page_in_use(cuda_ok):
    """The scale that a page already has counts as before, and a raised one rounds the page's tokens again."""
    w = near_ties.near([3.5], 5, 64)
    x = rows_of(w, E4M3)
    k = torch.from_numpy(x).to(torch.bfloat16).cuda()
    B = len(w)
    for first in (0.5, 3.0, 100.0):
        cache = Cache([2] * B, 16, 2, E4M3)
        held = torch.full((B, 2, 128), first, dtype=torch.bfloat16).cuda()
        cache.append(held, held, [0] * B)
        cache.append(k, k, [1] * B, inv_freq=torch.ones(8, dtype=torch.float64).cuda(), rot_offset=8,
                     rope_pos=torch.from_numpy(w[:, 0].astype(np.int32)).cuda())
        ok()
        got, _, ks, _ = cache.cpu()
        pid = cache.table[:, 0].long()
        y, _ = near_ties.turned(w[:, 0], w[:, 1], w[:, 2])
        e0 = ref.exponent(first, E4M3)
        want = np.array([2.0 ** max(e0, ref.exponent(float(abs(v)), E4M3)) for v in y])
        assert np.array_equal(ks[pid, 1].double().numpy(), want)
        once = ref.round8(first / 2.0 ** e0, E4M3) * 2.0 ** e0
        assert np.array_equal(got[pid, 0, 1].double().numpy(), np.repeat(ref.round8(once / want, E4M3)[:, None], 128, 1))
