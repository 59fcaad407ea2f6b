"""Infinities and NaN among rotated keys: each stored as the formula's own result."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from test_gpu_paged import Cache, E4M3, INT8, dsa

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("per", [1, 6])
def test_turned_infinities(cuda_ok, fmt, inter, per):
    """An infinite member of a pair at position 0 (sine 0) leaves (inf, NaN), or (NaN, inf); at others two infinities.
    The largest value stands for infinity; NaN stays NaN in e4m3 and becomes 0, reported, in int8."""
    pairs = [(INF, 2.0), (-INF, 2.0), (2.0, INF), (2.0, -INF), (INF, INF), (float("nan"), 1.0), (3.0, 2.0)]
    top = ref.TOP[fmt]
    one = lambda i: 2 * i if inter else i  # noqa: E731
    two = lambda i: 2 * i + 1 if inter else 32 + i  # noqa: E731
    for p in (0, 1, 5):
        c, s = np.cos(np.float64(p)), np.sin(np.float64(p))
        for a, b in pairs:
            x = torch.zeros((per, 1, 128), dtype=torch.bfloat16)
            x[:, 0, 64:] = 1.0
            x[per - 1, 0, one(9)], x[per - 1, 0, two(9)] = a, b
            x[per - 1, 0, one(4)], x[per - 1, 0, two(4)] = 1.5, -2.0
            pos = torch.zeros(per, dtype=torch.int32)
            pos[per - 1] = p
            cache = Cache([per], 16, 1, fmt)
            cache.append(x.cuda(), torch.ones_like(x).cuda(), [0], None if per == 1 else [per],
                         inv_freq=torch.ones(32, dtype=torch.float64).cuda(), interleaved=inter, rope_pos=pos.cuda())
            with np.errstate(invalid="ignore"):
                y = np.array([a * c - b * s, a * s + b * c])
            st = dsa.sync_status()
            assert st == (dsa.DSA_ERR_DEVICE_INPUT if fmt == INT8 and np.isnan(y).any() else dsa.DSA_OK), (p, a, b)
            k, _, ks, _ = cache.cpu()
            pid = int(cache.table[0, 0])
            others = [1.0, abs(1.5 * c + 2.0 * s), abs(1.5 * s - 2.0 * c)]
            scale = 2.0 ** ref.exponent(max([v for v in np.abs(y) if np.isfinite(v)] + others), fmt)
            assert float(ks[pid, 0]) == scale, (p, a, b)
            got = k[pid, per - 1, 0].double().numpy()
            for g, v in zip((got[one(9)], got[two(9)]), y):
                if np.isnan(v):
                    assert np.isnan(g) if fmt == E4M3 else g == 0, (p, a, b)
                else:
                    assert g == (np.sign(v) * top if np.isinf(v) else ref.round8(v / scale, fmt)), (p, a, b)
            rest = [ref.round8(v / scale, fmt) for v in (1.5 * c + 2.0 * s, 1.5 * s - 2.0 * c)]
            assert [got[one(4)], got[two(4)]] == rest, (p, a, b)
