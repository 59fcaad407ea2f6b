"""Attention over pages whose V scales lie as far apart as an append can leave them."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from test_gpu_paged import Cache, E4M3, INT8, check_attn, randn

pytestmark = pytest.mark.gpu


def pages_of(pattern, Hkv, fmt, page=16, seed=0):
    """A sequence whose pages hold random values with the V scales 2^pattern[i]; its keys tell pages with the smallest
    scale from the others: their dim 0 is 1, the others' 0, and all other dims 0.  (2^-2000 is 0.)"""
    n = len(pattern) * page
    cache = Cache([n], page, Hkv, fmt, seed=seed)
    rng = np.random.RandomState(seed)
    k, v, ks, vs = cache.cpu()
    for i, e in enumerate(pattern):
        pid = int(cache.table[0, i])
        kk = np.zeros((page, Hkv, 128))
        kk[..., 0] = e == min(pattern)
        k[pid] = torch.from_numpy(kk).to(fmt)
        v[pid] = torch.from_numpy(ref.round8(rng.uniform(20, 100, (page, Hkv, 128)), fmt)).to(fmt)
        ks[pid], vs[pid] = 1.0, 2.0 ** e
    for a, b in zip((cache.k, cache.v, cache.ks, cache.vs), (k, v, ks, vs)):
        a.copy_(b)
    return cache, n


PATTERNS = {
    "neighbours": [-64, 63], "in one step, reversed": [100, -64], "other warps": [-64, -64, 70, 70, -64, -64, 119, 119],
    "an ordinary page": [-6, 119, -6, -6], "rising": list(range(-64, 120, 20)), "falling": list(range(110, -65, -12)),
    "least": [-80] * 7, "least and most": [-80, 40, -80, 40, 0], "zeros among ordinary": [-64, -5, -64, -5, -5, -64] * 9,
    "long rows, halves": [-64] * 250 + [100] * 250, "long rows, halves reversed": [100] * 250 + [-64] * 250,
    "long rows, one": [-64] * 499 + [110],
    "scales of 0": [-2000, 100, -2000, 100, 100, -2000, -5],
}


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,G", [(4, 8), (1, 16)])
@pytest.mark.parametrize("name", PATTERNS)
def test_far_scales(cuda_ok, name, Hkv, G, fmt):
    """Rows whose logits are equal, and rows that lift the small pages' keys by 20, 60 and 100 nats or push them down:
    out and lse as in 64 bits, however little the small pages add to out."""
    cache, n = pages_of(PATTERNS[name], Hkv, fmt)
    lift = [0.0, 20.0, 60.0, 100.0, -20.0]
    q = torch.zeros((len(lift), Hkv * G, 128), dtype=torch.bfloat16)
    q[..., 0] = torch.tensor(lift)[:, None]
    q[..., 1:] = randn(3, len(lift), Hkv * G, 127)
    seq = [0] * len(lift)
    check_attn(cache, q, [n] * len(lift), 1.0, seq=seq)
    idx = np.stack([np.random.RandomState(i).permutation(n) for i in range(len(lift))])
    check_attn(cache, q, [n] * len(lift), 1.0, seq=seq, idx=idx)
