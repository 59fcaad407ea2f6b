"""Many keys of little weight beside one of nearly all of it: their part of the output is kept."""
import numpy as np
import pytest
import torch

from test_gpu_paged import Cache, E4M3, INT8, attend, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("selected", [False, True], ids=["dense", "selected"])
@pytest.mark.parametrize("Hkv,G,rows", [(4, 8, 200), (2, 16, 300), (1, 1, 1)])
def test_small_weights_are_not_lost(cuda_ok, Hkv, G, rows, selected, fmt):
    """One key's logit lies 25.5 binary orders above those of all others, whose values are 1 where its own are 0: the
    output is their share of the softmax.  A probability is off by 2^-32 of the largest (fp16 below 2^-21 of it),
    and by 2^-11 + 2^-20 of itself, the output by half a step more."""
    n = 49152 if rows > 1 else 6000
    cache = Cache([n], 128, Hkv, fmt)
    one = torch.ones((), dtype=fmt) if fmt == INT8 else torch.tensor(1.0).to(fmt)
    used = cache.table[0].long().cuda()
    cache.k.view(torch.uint8)[used] = 0
    cache.v.view(torch.uint8)[used] = one.view(torch.uint8).cuda()
    cache.ks[used], cache.vs[used] = 1.0, 1.0
    for at in (0, n // 2):
        pid, slot = int(cache.table[0, at // 128]), at % 128
        cache.k.view(torch.uint8)[pid, slot] = one.view(torch.uint8).cuda()
        cache.v.view(torch.uint8)[pid, slot] = 0
        q = torch.zeros((rows, Hkv * G, 128), dtype=torch.bfloat16)
        q[..., 3] = 25.5
        idx = None
        if selected:
            idx = torch.arange(n, dtype=torch.int32).expand(rows, n).contiguous()
        out, lse = attend(cache, q, [n] * rows, np.log(2.0), seq=[0] * rows, idx=idx)
        ok()
        rest = (n - 1) * 2.0 ** -25.5
        want = rest / (1 + rest)
        tol = want * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -18) + n * 2.0 ** -32
        assert tol < 0.05 * want
        assert (out.double() - want).abs().max() <= tol
        # the sum: a lane adds one of eight keys of a warp, which has a third of the row's at most, in fp32 to the large
        # key's weight; each addition is off by 2^-24 of the sum, n / 24 of them by n / 24 * 2^-24.  (The small weights
        # of that lane, 2^-25.5 of the large one's each, are below half its last bit, and all lost: that is the bound's
        # case.)  2^-18 (1 + lse) for the logits, their reference and the logarithm, as everywhere.
        wlse = 25.5 * np.log(2.0) + np.log1p(rest)
        assert (lse.double() - wlse).abs().max() <= n / 24 * 2.0 ** -24 + 2.0 ** -18 * (1 + wlse)
        cache.k.view(torch.uint8)[pid, slot] = 0
        cache.v.view(torch.uint8)[pid, slot] = one.view(torch.uint8).cuda()
