"""Rotated keys' bytes are those of the exact products; copied dims are copied."""
import numpy as np
import pytest
import torch

import near_ties
import paged_ref as ref
from test_gpu_paged import Cache, E4M3, INT8, dsa, ok, randn

pytestmark = pytest.mark.gpu


def ties(fmt):
    """Values halfway between two of the format's, of its normal range."""
    if fmt == INT8:
        return np.arange(8, 127) + 0.5
    return np.concatenate([(np.arange(8, 16) + 0.5) * 2.0 ** k for k in range(-6, 4)])


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("form", ["one token each", "long", "ragged"])
def test_bytes_next_to_a_tie(cuda_ok, fmt, inter, form):
    """Turned keys within 2^-23 of the middle between two bytes: rounding the fp32 rotation, right to 2^-24, would get
    many of them wrong, and the exact product gets all of them right."""
    count = 600
    w = near_ties.near(np.concatenate([ties(fmt), -ties(fmt)]), 11, count)
    y, z = near_ties.turned(w[:, 0], w[:, 1], w[:, 2])
    want, want2 = ref.round8(y.astype(np.float64), fmt), ref.round8(z.astype(np.float64), fmt)
    c, s = np.cos(w[:, 0]).astype(np.float32), np.sin(w[:, 0]).astype(np.float32)
    plain = w[:, 1].astype(np.float32) * c - w[:, 2].astype(np.float32) * s
    assert (ref.round8(plain.astype(np.float64), fmt) != want).sum() > count // 20
    i = np.arange(count)
    at = i % 16                                                      # the pair, of 16; turned dims 32 .. 63
    one, two = (32 + 2 * at, 33 + 2 * at) if inter else (32 + at, 48 + at)
    x = np.zeros((count, 1, 128))
    x[i, 0, one], x[i, 0, two] = w[:, 1], w[:, 2]
    x[:, 0, 0] = ref.TOP[fmt]                                        # the scale: 1
    k = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(k.double().numpy(), x)
    new = {"one token each": [1] * count, "long": [count], "ragged": [1, 30, 0, 65, 4, 500]}[form]
    assert sum(new) == count
    cache = Cache(new, 64, 1, fmt)
    cache.append(k.cuda(), k.cuda(), [0] * len(new), None if form == "one token each" else new,
                 inv_freq=torch.ones(16, dtype=torch.float64).cuda(), rot_offset=32, interleaved=inter,
                 rope_pos=torch.from_numpy(w[:, 0].astype(np.int32)).cuda())
    ok()
    pages, _, ks, _ = cache.cpu()
    seq = np.repeat(np.arange(len(new)), new)
    slot = np.concatenate([np.arange(n) for n in new])
    pid = cache.table.numpy()[seq, slot // 64]
    assert np.all(ks.numpy()[pid, 0] == 1.0)
    got = pages.double().numpy()[pid, slot % 64, 0]
    # the second members may come near a tie of their own: within 2^-30 either neighbour will do
    lo, hi = (ref.round8(z.astype(np.float64) * (1 + d), fmt) for d in (-2.0 ** -30, 2.0 ** -30))
    assert np.array_equal(got[i, one], want)
    assert np.all((got[i, two] == want2) | (got[i, two] == lo) | (got[i, two] == hi))


@pytest.mark.parametrize("R,off,inter", [(128, 0, False), (64, 32, True), (48, 40, False), (112, 8, True), (16, 112, False),
                                         (80, 48, True)])
@pytest.mark.parametrize("page,Hkv,fmt", [(64, 4, E4M3), (16, 2, INT8), (128, 1, E4M3)])
def test_bytes_of_random_keys(cuda_ok, page, Hkv, fmt, R, off, inter):
    """Every byte of ordinary keys is the exact product's.  The angle's own error (2^-52 of its size: the frequency's
    and 1 / 2 pi's roundings; 2^-61 a position: the turn's last bit) and fp64's roundings (2^-50) move the product by
    d; both ends of its interval are allowed, which differ where a tie lies within it."""
    n, new = 3000, [1000, 37, 1963]
    f, m = dsa.rope_freqs(R, 1e6, "yarn", 8.0, 32768)
    pos = np.random.RandomState(R).randint(0, 1 << 17, n)
    k = randn(R, n, Hkv, 128) * torch.exp2(randn(R + 1, n, 1, 1) * 2).to(torch.bfloat16)
    cache = Cache(new, page, Hkv, fmt)
    cache.append(k.cuda(), k.cuda(), [0] * 3, new, inv_freq=f.cuda(), mscale=m, rot_offset=off, interleaved=inter,
                 rope_pos=torch.from_numpy(pos.astype(np.int32)).cuda())
    ok()
    pages, _, ks, _ = cache.cpu()
    y, size, far = ref.rope(k.double().numpy(), pos, f.numpy(), off, inter, float(np.float32(m)))
    seq = np.repeat(np.arange(3), new)
    slot = np.concatenate([np.arange(x) for x in new])
    pid = cache.table.numpy()[seq, slot // page]
    s = ks.double().numpy()[pid][:, :, None]
    d = size * (far * 2.0 ** -52 + pos[:, None, None] * 2.0 ** -61 + 2.0 ** -50)
    got = pages.double().numpy()[pid, slot % page]
    assert np.all((got == ref.round8((y - d) / s, fmt)) | (got == ref.round8((y + d) / s, fmt)))
    assert (ref.round8((y - d) / s, fmt) != ref.round8((y + d) / s, fmt)).sum() < 10


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("D,R,off", [(64, 16, 0), (128, 64, 64), (192, 64, 120), (128, 128, 0), (512, 256, 8)])
def test_rope_turns_its_dims_and_no_others(cuda_ok, D, R, off, inter, dtype):
    """Half a turn a position: at odd positions exactly the R turned dims change sign (to 2^-20), all others stay."""
    x = randn(D, 5, 3, D, dtype=dtype).abs() + 1
    f = torch.full((R // 2,), np.pi, dtype=torch.float64).cuda()
    out = torch.empty((5, 3, D), dtype=dtype, device="cuda")
    dsa.dsa_rope(x.to(dtype).cuda(), out, f, rot_offset=off, interleaved=inter)
    ok()
    turned = (out.cpu() < 0).sum((1, 2))
    assert turned.tolist() == [0, 3 * R, 0, 3 * R, 0]
    rest = torch.ones(D, dtype=torch.bool)
    rest[off:off + R] = False
    assert torch.equal(out.cpu()[..., rest], x.to(dtype)[..., rest])
