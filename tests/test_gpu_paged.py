"""Rotary positions, the paged 8-bit cache's append and the attention over that cache on a GPU, against
their definitions in 64 bits (paged_ref)."""
import numpy as np
import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("dsa_lightning_indexer_02_b200")

BF, FP32 = torch.bfloat16, torch.float32
E4M3, INT8 = ref.E4M3, ref.INT8


def ok():
    assert dsa.sync_status() == dsa.DSA_OK


def randn(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


# ------------------------------------------------------------------ rotary positions
def rope_bound(y, size, far, dtype):
    """bf16: the sine and cosine are off by 2^-21 each and two products and a sum by 2^-24 each, then half a
    step; fp32: sine and cosine by 2 ulp, their factor, the products and the sum by half an ulp each.  The
    angle itself is off by 2^-52 of its size (and by 2^-30 for its last kept bit)."""
    angle = far * 2.0 ** -52 + 2.0 ** -29
    return size * ((2.0 ** -20 if dtype == BF else 2.0 ** -21) + angle) + (2.0 ** -8 * np.abs(y) if dtype == BF else 0) + 1e-38


ROPE = [
    # T, H, D, R, off, pos0 or "random"
    (1, 1, 64, 16, 0, 0), (1, 32, 128, 128, 0, 131071), (3, 5, 128, 64, 64, "random"), (257, 4, 64, 32, 32, 77),
    (130, 2, 192, 64, 128, "random"), (40, 7, 8 * 3, 16, 8, -5), (19, 3, 512, 256, 128, 1 << 30),
    (1000, 1, 128, 96, 16, "random"), (5, 300, 64, 64, 0, 9),
]


@pytest.mark.parametrize("dtype", [BF, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,R,off,pos", ROPE)
def test_rope(cuda_ok, T, H, D, R, off, pos, inter, dtype):
    x = randn(T + H, T, H, D, dtype=dtype)
    f, m = dsa.rope_freqs(R, 1e4, "yarn", 4.0, 4096)
    p = None
    where = np.arange(T, dtype=np.int64) + (pos if pos != "random" else 0)
    if pos == "random":
        where = np.random.RandomState(T).randint(-2 ** 31, 2 ** 31, T)
        p = torch.from_numpy(where.astype(np.int32)).cuda()
    for inverse in (False, True):
        out = torch.full((T, H, D), float("nan"), dtype=dtype, device="cuda")
        dsa.dsa_rope(x.cuda(), out, f.cuda(), pos=p, pos0=0 if p is not None else pos, rot_offset=off, interleaved=inter,
                     mscale=m, inverse=inverse)
        ok()
        y, size, far = ref.rope(x.double().numpy(), where, f.numpy(), off, inter, m, inverse)
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - y) <= rope_bound(y, size, far, dtype))
        still = size[0, 0] == 0
        assert np.array_equal(got[..., :off], x.double().numpy()[..., :off])
        assert np.array_equal(got[..., off + R:], x.double().numpy()[..., off + R:]) and still.sum() <= D


@pytest.mark.parametrize("dtype", [BF, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
def test_rope_strides_in_place_and_broadcast(cuda_ok, inter, dtype):
    T, H, D, R = 77, 6, 128, 64
    f, _ = dsa.rope_freqs(R, 1e6)
    f = f.cuda()
    kw = dict(pos0=100, rot_offset=32, interleaved=inter)
    wide = randn(1, T, 10 * D, dtype=dtype).cuda()
    x = wide[:, 2 * D:8 * D].unflatten(1, (H, D))                   # heads of a fused projection
    want = torch.empty((T, H, D), dtype=dtype, device="cuda")
    dsa.dsa_rope(x.contiguous(), want, f, **kw)
    by_head = torch.zeros((H, T, D + 8), dtype=dtype, device="cuda")
    dsa.dsa_rope(x, by_head.transpose(0, 1)[..., :D], f, **kw)      # heads before tokens, padded rows
    assert torch.equal(by_head.transpose(0, 1)[..., :D], want) and not by_head[..., D:].any()
    one = x[:1].expand(T, H, D)                                     # one token's row at every position
    got = torch.empty_like(want)
    dsa.dsa_rope(one, got, f, **kw)
    also = torch.empty_like(want)
    dsa.dsa_rope(one.contiguous(), also, f, **kw)
    assert torch.equal(got, also)
    rest = wide.clone()
    dsa.dsa_rope(x, x, f, **kw)                                     # in place inside the projection
    ok()
    assert torch.equal(x, want)
    assert torch.equal(wide[:, :2 * D], rest[:, :2 * D]) and torch.equal(wide[:, 8 * D:], rest[:, 8 * D:])


def test_rope_copies_bits_and_turns_infinities(cuda_ok):
    """Dims outside the rotated ones keep their bits, NaN and infinities among them, and those inside give
    what the formula gives."""
    x = torch.zeros((1, 1, 64), dtype=BF)
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2], x[0, 0, 40] = float("nan"), float("inf"), -0.0, float("inf")
    x[0, 0, 48:] = torch.tensor([float("nan"), -0.0] * 8)
    f, _ = dsa.rope_freqs(32)
    out = torch.empty((1, 1, 64), dtype=BF, device="cuda")
    dsa.dsa_rope(x.cuda(), out, f.cuda(), pos0=3, rot_offset=16)
    ok()
    got = out.cpu()
    assert torch.equal(got[..., :16].view(torch.int16), x[..., :16].view(torch.int16))
    assert torch.equal(got[..., 48:].view(torch.int16), x[..., 48:].view(torch.int16))
    assert torch.isinf(got[0, 0, 40]) and torch.isinf(got[0, 0, 24])   # pair 8: (24, 40)
    assert not torch.isnan(got[..., 16:48]).any()


def test_rope_gradient_against_differences(cuda_ok):
    """<g, R(x + e) - R(x - e)> / 2 e = <R'(g), x-direction>: the rotation is linear, so fp32 rounding alone
    separates the two (|sums| < 64 over 4096 products: 2^-10 leaves room)."""
    T, H, D, R = 8, 4, 128, 96
    f, m = dsa.rope_freqs(R, 1e4, "ntk", 8.0)
    f = f.cuda()
    x, d, g = (randn(s, T, H, D, dtype=FP32).cuda() for s in (1, 2, 3))
    grad = torch.empty_like(g)
    for inter in (False, True):
        kw = dict(pos0=12345, rot_offset=16, interleaved=inter, mscale=1.25)
        dsa.dsa_rope(g, grad, f, inverse=True, **kw)
        lo, hi = torch.empty_like(x), torch.empty_like(x)
        dsa.dsa_rope(x - d, lo, f, **kw)
        dsa.dsa_rope(x + d, hi, f, **kw)
        ok()
        num = ((hi.double() - lo.double()) / 2 * g.double()).sum()
        assert abs(num - (grad.double() * d.double()).sum()) <= 2.0 ** -10


# ------------------------------------------------------------------ cache
class Cache:
    """A pool of pages with a table that deals them to sequences of up to the given capacities in any order.
    Unwritten bytes are NaN in e4m3 (-128 in int8), unwritten scales NaN, free table entries -1."""

    def __init__(self, caps, page, Hkv, fmt, seed=0, spare=2):
        self.page, self.fmt, self.Hkv = page, fmt, Hkv
        per = [-(-c // page) for c in caps]
        order = np.random.RandomState(seed).permutation(sum(per) + spare)
        self.table = torch.full((len(caps), max(max(per), 1)), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(per):
            self.table[b, :k] = torch.from_numpy(order[at:at + k].astype(np.int32))
            at += k
        num = sum(per) + spare
        raw = torch.full((num, page, Hkv, 128), 0x7f if fmt == E4M3 else 0x80, dtype=torch.uint8)
        self.k, self.v = raw.view(fmt).cuda(), raw.clone().view(fmt).cuda()
        self.ks = torch.full((num, Hkv), float("nan"), device="cuda")
        self.vs = self.ks.clone()
        self.table_gpu = self.table.cuda()

    def append(self, k, v, ctx, new=None, **kw):
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        cu = None if new is None else i32([0] + list(np.cumsum(new)))
        dsa.dsa_kv_append(k, v, self.k, self.v, self.ks, self.vs, self.table_gpu, i32(ctx), cu_new=cu, **kw)

    def cpu(self):
        return [t.cpu() for t in (self.k, self.v, self.ks, self.vs)]


def check_append(before, after, table, page, fmt, ctx, new, x, err, name):
    """`after` against the definition: x float64 [N, Hkv, 128] as it is to be stored, err its allowed error."""
    (pages0, scale0), (pages1, scale1) = before, after
    pages0, pages1 = pages0.double().numpy(), pages1.double().numpy()
    scale0, scale1 = scale0.double().numpy(), scale1.double().numpy()
    touched = np.zeros(pages1.shape[:2], dtype=bool)
    scaled = np.zeros(scale1.shape, dtype=bool)
    i = 0
    for b, n in enumerate(new):
        c = ctx[b]
        end = i + n
        while i < end:
            pid, slot = int(table[b, c // page]), c % page
            k = min(end - i, page - slot)
            for h in range(x.shape[1]):
                xs = x[i:i + k, h]
                need = 2.0 ** ref.exponent(np.abs(xs).max(), fmt)
                s = max(need, scale0[pid, h]) if slot else need
                assert scale1[pid, h] == s, (name, b, c, h)
                got, y = pages1[pid, slot:slot + k, h], xs / s
                if err is None:
                    assert np.array_equal(got, ref.round8(y, fmt)), (name, b, c, h)
                else:
                    assert np.all(np.abs(got - y) <= 0.5 * ref.step8(np.abs(y) + err[i:i + k, h] / s, fmt) + err[i:i + k, h] / s)
                if slot:
                    held = ref.round8(pages0[pid, :slot, h] * (scale0[pid, h] / s), fmt)
                    assert np.array_equal(pages1[pid, :slot, h], held), (name, b, c, h)
                scaled[pid, h] = True
            touched[pid, :slot + k] = True
            i, c = i + k, c + k
    # everything else as it was, bit for bit
    raw0, raw1 = (np.nan_to_num(p, nan=1e9) for p in (pages0, pages1))
    assert np.array_equal(raw0[~touched], raw1[~touched]), name
    assert np.array_equal(np.isnan(scale1), ~scaled & np.isnan(scale0)) and \
        np.array_equal(scale1[~scaled & ~np.isnan(scale0)], scale0[~scaled & ~np.isnan(scale0)]), name


APPEND = [
    # page, Hkv, fmt, tokens of each step for each sequence
    (16, 1, E4M3, [[0, 1, 15, 16, 17, 40], [1, 0, 1, 16, 15, 3], [30, 2, 0, 0, 1, 5]]),
    (64, 4, E4M3, [[63, 64, 65, 1, 0, 200], [1, 1, 1, 1, 1, 1], [2, 70, 0, 129, 63, 9]]),
    (32, 2, INT8, [[31, 33, 0, 5], [1, 1, 1, 1], [64, 1, 7, 32]]),
    (128, 4, INT8, [[300, 1, 0], [1, 127, 128], [1, 1, 1]]),
    (128, 1, E4M3, [[5], [123], [1], [260]]),
    # sequences enough that a thread takes four rows, not two
    (64, 4, E4M3, [[i % 70 for i in range(150)], [i * 7 % 66 for i in range(150)]]),
    (16, 2, INT8, [[i % 19 for i in range(700)], [i * 5 % 18 for i in range(700)]]),
    (128, 1, E4M3, [[i * 3 % 131 for i in range(90)], [i % 60 for i in range(90)]]),
]


@pytest.mark.parametrize("R,off,inter", [(0, 0, False), (128, 0, False), (32, 96, False), (64, 16, True)],
                         ids=["plain", "half", "part", "interleaved"])
@pytest.mark.parametrize("page,Hkv,fmt,steps", APPEND)
def test_append(cuda_ok, page, Hkv, fmt, steps, R, off, inter):
    """Step after step into the same cache, magnitudes growing and falling, so that scales of partly
    filled pages grow and held tokens are rounded again."""
    B = len(steps[0])
    cache = Cache([sum(s[b] for s in steps) for b in range(B)], page, Hkv, fmt, seed=page)
    ctx = [0] * B
    f, m = dsa.rope_freqs(R, 1e4, "yarn", 4.0, 4096) if R else (None, 1.0)
    for i, new in enumerate(steps):
        n = sum(new)
        kv = randn(i, n, 2 * Hkv + 1, 128) * torch.exp2(randn(i + 9, n, 1, 1) * 2 + 3 * (i % 2)).to(BF)
        k, v = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]                       # slices of one projection
        pos = np.concatenate([c + np.arange(x) for c, x in zip(ctx, new)] or [[]])
        before = cache.cpu()
        rot = dict(inv_freq=f.cuda(), rot_offset=off, interleaved=inter, mscale=m) if R else {}
        if R == 32:                                                # positions other than the cache's
            pos = np.random.RandomState(i).randint(0, 1 << 20, n)
            rot["rope_pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        gpu = kv.cuda()
        cache.append(gpu[:, :Hkv], gpu[:, Hkv:2 * Hkv], ctx, None if set(new) == {1} else new, **rot)
        ok()
        after = cache.cpu()
        kd, err = k.double().numpy(), None
        if R:
            kd, size, far = ref.rope(kd, pos, f.numpy(), off, inter, m)
            err = rope_bound(kd, size, far, FP32)
        check_append((before[0], before[2]), (after[0], after[2]), cache.table, page, fmt, ctx, new, kd, err, "k")
        check_append((before[1], before[3]), (after[1], after[3]), cache.table, page, fmt, ctx, new,
                     v.double().numpy(), None, "v")
        ctx = [c + x for c, x in zip(ctx, new)]


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
def test_append_extreme_values(cuda_ok, fmt):
    """Zeros, the format's exact bounds, bf16's largest, subnormals, infinities and NaN."""
    top = ref.TOP[fmt]
    big = float(torch.finfo(BF).max)
    rows = [0.0, top * 8, top * 8 + (32 if fmt == E4M3 else 8), big, 1e-39, 2.0 ** -64, float("inf"), -float("inf")]
    x = torch.zeros((len(rows), 1, 128), dtype=BF)
    for i, r in enumerate(rows):
        x[i, 0, 5] = r
        x[i, 0, 7] = 1.0 if np.isinf(r) else r / 3
    cache = Cache([1] * len(rows), 16, 1, fmt)
    cache.append(x.cuda(), x.cuda(), [0] * len(rows))
    ok()
    k, v, ks, vs = cache.cpu()
    for i, r in enumerate(rows):
        pid = int(cache.table[i, 0])
        finite = np.nan_to_num(x[i, 0].double().numpy(), posinf=0, neginf=0)
        e = ref.exponent(np.abs(finite).max(), fmt)
        assert ks[pid, 0] == vs[pid, 0] == 2.0 ** e
        want = ref.round8(np.clip(x[i, 0].double().numpy() / 2.0 ** e, -1e9, 1e9), fmt)
        for t in (k, v):
            assert np.array_equal(t[pid, 0, 0].double().numpy(), want), r
    # NaN: kept by e4m3, 0 and reported in int8; the block's other values as without it
    cache = Cache([1], 16, 1, fmt)
    x = torch.full((1, 1, 128), 3.0, dtype=BF)
    x[0, 0, 9] = float("nan")
    cache.append(x.cuda(), x.cuda(), [0])
    assert dsa.sync_status() == (dsa.DSA_OK if fmt == E4M3 else dsa.DSA_ERR_DEVICE_INPUT)
    k, v, ks, _ = cache.cpu()
    got = k[int(cache.table[0, 0]), 0, 0].double()
    assert torch.isnan(got[9]) if fmt == E4M3 else got[9] == 0
    got[9] = 3.0 / float(ks[int(cache.table[0, 0]), 0])
    assert torch.all(got * ks[int(cache.table[0, 0]), 0].double() == 3.0)


def test_append_restarts_recycled_pages_and_rolls_back(cuda_ok):
    """A page of a finished sequence, given to another, starts anew with its slot 0; after a rollback within
    a page its scale stays at least what the kept tokens need."""
    cache = Cache([64], 64, 1, E4M3, spare=0)
    big, small = torch.full((10, 1, 128), 1000.0, dtype=BF), torch.full((4, 1, 128), 0.01, dtype=BF)
    cache.append(big.cuda(), big.cuda(), [0], [10])
    assert cache.cpu()[2][0, 0] == 2.0 ** ref.exponent(1000.0, E4M3)
    cache.append(small.cuda(), small.cuda(), [5], [4])               # five of the ten taken back
    assert cache.cpu()[2][0, 0] == 2.0 ** ref.exponent(1000.0, E4M3)
    cache.append(small.cuda(), small.cuda(), [0], [4])               # the page recycled
    ok()
    k, _, ks, _ = cache.cpu()
    s = 2.0 ** ref.exponent(float(small[0, 0, 0]), E4M3)
    assert ks[0, 0] == s and torch.all(k[0, :4].double() == ref.round8(float(small[0, 0, 0]) / s, E4M3).item())


def test_append_bad_device_inputs_are_skipped_and_reported(cuda_ok):
    """A context beyond the table, a negative one, token ranges outside k_new and page numbers outside the pool:
    those sequences (pages) are left as they were, the others are appended, and the call is reported."""
    def run(ctx, cu, n, spoil=None):
        cache = Cache([32, 32, 32], 16, 1, E4M3)
        if spoil is not None:
            cache.table_gpu[1, 0] = spoil
        x = torch.full((n, 1, 128), 2.0, dtype=BF).cuda()
        dsa.dsa_kv_append(x, x, cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu,
                          torch.tensor(ctx, dtype=torch.int32).cuda(), cu_new=torch.tensor(cu, dtype=torch.int32).cuda())
        st = dsa.sync_status()
        k = cache.cpu()[0]
        written = [int((~torch.isnan(k[cache.table[b].long()].double())).sum()) // 128 for b in range(3)]
        return st, written

    assert run([0, 0, 0], [0, 2, 4, 6], 6) == (dsa.DSA_OK, [2, 2, 2])
    assert run([0, 31, 0], [0, 2, 4, 6], 6) == (dsa.DSA_ERR_DEVICE_INPUT, [2, 0, 2])
    assert run([0, -1, 0], [0, 2, 4, 6], 6) == (dsa.DSA_ERR_DEVICE_INPUT, [2, 0, 2])
    assert run([0, 0, 0], [0, 2, 4, 9], 6) == (dsa.DSA_ERR_DEVICE_INPUT, [2, 2, 0])
    assert run([0, 0, 0], [0, 2, 20, 6], 6)[0] == dsa.DSA_ERR_DEVICE_INPUT
    assert run([0, 0, 0], [0, 20, 22, 24], 24, spoil=-1) == (dsa.DSA_ERR_DEVICE_INPUT, [20, 0, 2])
    assert run([0, 0, 0], [0, 20, 22, 24], 24, spoil=1000) == (dsa.DSA_ERR_DEVICE_INPUT, [20, 0, 2])
    assert run([0, 0, 0], [1, 2, 4, 5], 6) == (dsa.DSA_OK, [1, 2, 1])     # tokens outside the ranges are ignored


# ------------------------------------------------------------------ attention
def filled(lens, page, Hkv, fmt, seed=0, spread=1.0):
    """A cache with random tokens, scales of any power of two within 2^(+-spread)."""
    cache = Cache(lens, page, Hkv, fmt, seed=seed)
    rng = np.random.RandomState(seed + 1)
    k, v, ks, vs = cache.cpu()
    for b, n in enumerate(lens):
        for p in range(-(-n // page)):
            pid, m = int(cache.table[b, p]), min(page, n - p * page)
            for pages, scale, size in ((k, ks, 1.0), (v, vs, 2.0)):
                x = rng.standard_normal((m, Hkv, 128)) * (100 if fmt == E4M3 else 30)
                pages[pid, :m] = torch.from_numpy(ref.round8(x, fmt)).to(fmt)
                scale[pid] = torch.from_numpy(2.0 ** (np.round(rng.uniform(-spread, spread, Hkv)) - (6.0 if fmt == E4M3 else 5.0)))
    for a, b in zip((cache.k, cache.v, cache.ks, cache.vs), (k, v, ks, vs)):
        a.copy_(b)
    return cache


def attend(cache, q, n_keys, scale=128 ** -0.5, seq=None, idx=None, **kw):
    q = q.cuda()
    i32 = lambda a: None if a is None else torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    dsa.dsa_paged_attn(q, cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu, i32(n_keys), scale, out, seq=i32(seq),
                       idx=i32(idx), lse=lse, **kw)
    return out, lse


def check_attn(cache, q, n_keys, scale=128 ** -0.5, seq=None, idx=None):
    out, lse = attend(cache, q, n_keys, scale, seq, idx)
    ok()
    want, wlse, tol, ltol = ref.attn(q, *cache.cpu(), cache.table, n_keys, scale, seq, None if idx is None else np.asarray(idx))
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), np.nanmax(np.abs(got - want) / (tol + 1e-300))
    none = np.isinf(wlse)
    assert np.array_equal(glse[none], wlse[none])
    assert np.all(np.abs(glse[~none] - wlse[~none]) <= ltol[~none])
    again = attend(cache, q, n_keys, scale, seq, idx)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    return out


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,G,page,lens", [
    (1, 1, 16, [1]), (4, 8, 64, [0, 1, 2, 63, 64, 65, 300]), (2, 16, 16, [1000, 15, 0, 17]),
    (1, 16, 128, [129, 500]), (4, 7, 32, [33, 31, 2000]), (2, 5, 128, [700]), (4, 16, 64, [5, 640]),
    (1, 8, 32, [3001]), (4, 1, 16, [48, 47, 49]),
])
def test_attn_dense(cuda_ok, Hkv, G, page, lens, fmt):
    cache = filled(lens, page, Hkv, fmt, seed=Hkv * G)
    check_attn(cache, randn(G, len(lens), Hkv * G, 128), lens)


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,G", [(4, 8), (1, 16), (2, 3)])
def test_attn_many_rows_a_sequence(cuda_ok, Hkv, G, fmt):
    """Causal rows of three sequences (a chunk of 9, a chunk longer than its sequence, one alone), in any order."""
    lens = [100, 4, 333]
    cache = filled(lens, 16, Hkv, fmt, seed=3)
    seq = [0] * 9 + [1] * 6 + [2]
    n = [92 + i for i in range(9)] + [0, 0, 1, 2, 3, 4] + [333]
    order = np.random.RandomState(0).permutation(len(seq))
    check_attn(cache, randn(7, len(seq), Hkv * G, 128), np.array(n)[order], seq=np.array(seq)[order])


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,G,page", [(4, 8, 64), (2, 16, 16), (1, 4, 128)])
@pytest.mark.parametrize("topk", [1, 37, 512])
def test_attn_selected_keys(cuda_ok, Hkv, G, page, topk, fmt):
    """Rows with fewer keys than topk, holes, only -1, keys beyond the row's, repeated keys, no keys at all."""
    lens = [600, 40, 5, 0]
    cache = filled(lens, page, Hkv, fmt, seed=topk)
    seq = [0, 0, 1, 1, 2, 3, 0]
    n = [600, 77, 40, 13, 5, 0, 600]
    rng = np.random.RandomState(topk)
    idx = np.full((len(seq), topk), -1)
    for r, m in enumerate(n):
        k = min(topk, m)
        idx[r, :k] = rng.permutation(m)[:k]
    idx[1, ::3] = -1
    idx[2, ::2] = 40 + rng.randint(0, 1000, len(idx[2, ::2]))
    idx[3] = -1
    idx[4] = 4
    idx[6, : topk // 2] = idx[6, 0]
    check_attn(cache, randn(topk, len(seq), Hkv * G, 128), n, seq=seq, idx=idx)


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("spread,qs", [(30, 2.0 ** -20), (12, 2.0 ** -6), (1, 2.0 ** 60), (1, 2.0 ** -100)])
def test_attn_wide_scales(cuda_ok, spread, qs, fmt):
    """Blocks whose scales lie far apart (K's and V's), queries of any size, and scales that are no powers of two."""
    lens = [400, 70]
    cache = filled(lens, 16, 2, fmt, seed=5, spread=spread)
    q = (randn(1, 2, 16, 128, dtype=FP32) * qs).to(BF)
    scale = 128 ** -0.5 * (2.0 ** -60 if qs > 1e9 else 1.0)
    check_attn(cache, q, lens, scale)
    cache.ks *= 1.3
    cache.vs *= -0.7
    cache.vs[int(cache.table[0, 3])] = 0.0
    check_attn(cache, q, lens, scale)


def test_attn_many_rows_and_long_rows(cuda_ok):
    """Enough rows that each gets a block, and one long row that many blocks share, beside short ones."""
    cache = filled([3000], 64, 4, E4M3)
    rows = 3000
    n = np.random.RandomState(2).randint(0, 60, rows)
    q = randn(4, rows, 8, 128)
    check_attn(cache, q, n, seq=[0] * rows)
    cache = filled([20000, 3, 0, 700], 64, 1, INT8)
    check_attn(cache, randn(5, 4, 8, 128), [20000, 3, 0, 700])


def test_attn_reads_only_attended_slots(cuda_ok):
    """Slots behind a row's keys, pages of others and unused table entries hold NaN or -1: no result depends on
    them, and NaN in an attended key reaches just the rows that attend to it."""
    cache = filled([70, 50], 16, 2, E4M3, seed=8)
    q = randn(3, 4, 8, 128)
    args = dict(n_keys=[70, 33, 32, 50], seq=[0, 0, 0, 1])
    want = check_attn(cache, q, **args)
    pid = int(cache.table[0, 2])
    cache.v.view(torch.uint8)[pid, 0, 1, 5] = 0x7f                   # position 32 of sequence 0
    got, _ = attend(cache, q, **args)
    ok()
    bad = torch.isnan(got)
    assert bad[:2, 4:, 5].all() and bad.sum() == 8
    assert torch.equal(got[2:], want[2:]) and torch.equal(got[:, :4], want[:, :4])


def test_attn_bad_device_inputs_are_skipped_and_reported(cuda_ok):
    cache = filled([40, 40], 16, 1, E4M3)
    q = randn(2, 4, 4, 128)
    want, wl = attend(cache, q, [40, 40, 40, 40], seq=[0, 1, 0, 1])
    ok()
    for n, seq in (([40, 49, 40, 40], [0, 1, 0, 1]), ([40, -1, 40, 40], [0, 1, 0, 1]), ([40] * 4, [0, 2, 0, 1]),
                   ([40] * 4, [0, -1, 0, 1])):
        out, lse = attend(cache, q, n, seq=seq)
        assert dsa.sync_status() == dsa.DSA_ERR_DEVICE_INPUT
        assert not out[1].any() and torch.isinf(lse[1]).all()
        assert torch.equal(out[[0, 2, 3]], want[[0, 2, 3]])
    for page in (-1, 10 ** 6):
        cache.table_gpu[1, 1] = page                                 # keys 16 .. 31 of sequence 1
        out, _ = attend(cache, q, [40] * 4, seq=[0, 1, 0, 1])
        assert dsa.sync_status() == dsa.DSA_ERR_DEVICE_INPUT
        idx = np.tile(np.r_[0:16, 32:40, -np.ones(16)], (4, 1))
        idx[[0, 2]] = np.arange(40)
        cache.table_gpu[1, 1] = cache.table[1, 1]
        also, _ = attend(cache, q, [40] * 4, seq=[0, 1, 0, 1], idx=idx)
        ok()
        assert (out.double() - also.double()).abs().max() <= 2.0 ** -7 * also.double().abs().max()


def test_cache_beyond_four_gigabytes(cuda_ok):
    """Pages whose byte offsets pass 2^32: appended and read back through the attention."""
    page, Hkv, pages = 128, 4, 80000                                 # 5.2 GB for K and for V
    k = torch.empty((pages, page, Hkv, 128), dtype=E4M3, device="cuda")
    v = torch.empty_like(k)
    ks, vs = torch.zeros((pages, Hkv), device="cuda"), torch.zeros((pages, Hkv), device="cuda")
    small = Cache([200], page, Hkv, E4M3)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    x = randn(6, 200, 2 * Hkv, 128).cuda()
    q = randn(7, 1, 32, 128).cuda()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    dsa.dsa_kv_append(x[:, :Hkv], x[:, Hkv:], k, v, ks, vs, table, i32(0), cu_new=i32(0, 200))
    out = torch.empty_like(q)
    dsa.dsa_paged_attn(q, k, v, ks, vs, table, i32(200), 0.1, out)
    small.append(x[:, :Hkv], x[:, Hkv:], [0], [200])
    want, _ = attend(small, q.cpu(), [200], 0.1)
    ok()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ as they are used together
def test_serving_loop(cuda_ok):
    """A ragged prefill and three decode steps of a DSA decoder on the paged cache: rotate q, qI, kI; append; score,
    select and attend.  Against the same in 64 bits from the inputs on (keys as the cache holds them)."""
    B, Hq, Hkv, HI, topk, page = 3, 16, 2, 16, 48, 16
    lens, steps = [100, 7, 64], 3
    f, m = dsa.rope_freqs(64, 1e4, "yarn", 4.0, 64)
    fI, _ = dsa.rope_freqs(32, 1e4)
    fg, fIg = f.cuda(), fI.cuda()
    cache = Cache([n + steps for n in lens], page, Hkv, E4M3)
    kI_all = torch.zeros((B, 128, 64), dtype=BF, device="cuda")
    ctx = [0] * B
    for step in range(1 + steps):
        new = lens if step == 0 else [1] * B
        n = sum(new)
        pos = np.concatenate([c + np.arange(x) for c, x in zip(ctx, new)])
        posg = torch.from_numpy(pos.astype(np.int32)).cuda()
        qkv = randn(step, n, (Hq + 2 * Hkv) * 128).cuda()
        q, k, v = qkv.split([Hq * 128, Hkv * 128, Hkv * 128], 1)
        q, k, v = q.unflatten(1, (Hq, 128)), k.unflatten(1, (Hkv, 128)), v.unflatten(1, (Hkv, 128))
        qI, kI, w = randn(step + 50, n, HI, 64).cuda(), randn(step + 60, n, 1, 64).cuda(), randn(step + 70, n, HI).cuda()
        cache.append(k, v, ctx, new, inv_freq=fg, mscale=m)
        dsa.dsa_rope(q, q, fg, pos=posg, mscale=m)
        dsa.dsa_rope(qI, qI, fIg, pos=posg)
        dsa.dsa_rope(kI, kI, fIg, pos=posg)
        seq = np.repeat(np.arange(B), new)
        kI_all[torch.from_numpy(seq).cuda(), posg.long()] = kI[:, 0]
        idx = torch.empty((n, topk), dtype=torch.int32, device="cuda")
        i = 0
        for b in range(B):
            c, x = ctx[b], new[b]
            scores = torch.empty((x, (c + x + 3) // 4 * 4), device="cuda")
            dsa.dsa_index(qI[i:i + x].contiguous(), kI_all[b], w[i:i + x], c, scores)
            part = torch.empty((x, topk), dtype=torch.int32, device="cuda")
            dsa.dsa_topk(scores, c, topk, part)
            idx[i:i + x] = part
            i += x
        ok()
        check_attn(cache, q.cpu().contiguous(), pos + 1, seq=seq, idx=idx.cpu().numpy())
        # and near the attention over the unrounded keys and values of this step's tokens alone: one token
        # attending to itself returns its value, rounded to e4m3 (2^-4 of it, 2^-10 of the block's scale)
        out, _ = attend(cache, q.cpu().contiguous(), pos + 1, seq=seq, idx=pos[:, None])
        _, _, _, vs = cache.cpu()
        own = v.double().cpu().repeat_interleave(Hq // Hkv, 1)
        s = vs[cache.table[seq, pos // page].long()].double().repeat_interleave(Hq // Hkv, 1)[..., None]
        far = (out.double().cpu() - own).abs() > own.abs() * (2.0 ** -4 + 2.0 ** -8) + s * 2.0 ** -9
        assert not (far & torch.from_numpy(pos + 1 <= topk)[:, None, None]).any()
        ctx = [c + x for c, x in zip(ctx, new)]


def test_graph_replays_follow_their_inputs(cuda_ok):
    """Rotation, append and attention captured once and replayed step after step, lengths advanced on the device;
    two graphs with a workspace each, replayed on two streams at once."""
    def loop(graph):
        cache = Cache([40, 30], 16, 4, E4M3, seed=1)
        ctx = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
        n = torch.empty_like(ctx)
        x = torch.zeros((2, 40, 128), dtype=BF, device="cuda")
        first = randn(0, 3, 8, 128).cuda()
        i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        dsa.dsa_kv_append(first[:, :4], first[:, 4:], cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu, i32(0, 0),
                          cu_new=i32(0, 3, 3))
        f = dsa.rope_freqs(128)[0].cuda()
        q, out = torch.empty((2, 32, 128), dtype=BF, device="cuda"), torch.empty((2, 32, 128), dtype=BF, device="cuda")
        ws = torch.empty(dsa.workspace_size(dsa.DSA_OP_PAGED_ATTN, 1, 2, 32, 1, 1), dtype=torch.uint8, device="cuda")

        def step():
            dsa.dsa_rope(x[:, :32], q, f, pos=ctx)
            dsa.dsa_kv_append(x[:, 32:36], x[:, 36:], cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu, ctx, inv_freq=f)
            torch.add(ctx, 1, out=n)
            dsa.dsa_paged_attn(q, cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu, n, 0.09, out, ws=ws)
            ctx.copy_(n)

        if not graph:
            return x, out, step, step
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            step()
        return x, out, g.replay, step                                # step holds the captured tensors

    plain, graphs = loop(False), [loop(True), loop(True)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(20):
        x = randn(100 + i, 2, 40, 128).cuda()
        plain[0].copy_(x)
        plain[2]()
        torch.cuda.synchronize()
        for (xs, _, replay, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                xs.copy_(x)
                replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], plain[1]) and torch.equal(graphs[1][1], plain[1])
    ok()


def test_other_stream(cuda_ok):
    """Calls on a stream that is not the current one, their workspace among it."""
    s = torch.cuda.Stream()
    cache = filled([500, 20], 16, 4, E4M3)
    q = randn(0, 2, 32, 128).cuda()
    n = torch.tensor([500, 20], dtype=torch.int32, device="cuda")
    want, out = torch.empty_like(q), torch.empty_like(q)
    dsa.dsa_paged_attn(q, cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu, n, 0.1, want)
    torch.cuda.synchronize()
    for _ in range(20):
        dsa.dsa_paged_attn(q, cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu, n, 0.1, out, stream=s)
        torch.empty(20 << 20, dtype=torch.uint8, device="cuda").fill_(255)   # freed memory that a call must not share
    s.synchronize()
    ok()
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows,most", [(1, 64), (3, 200), (16, 800), (40, 800), (64, 800), (128, 200), (160, 640),
                                       (1, 4096), (5, 20000), (1184, 640), (1185, 64), (1, 288), (2, 480), (3, 576), (1, 672)])
def test_attn_every_spread_of_rows(cuda_ok, rows, most):
    """Row counts and table widths on both sides of each choice between dealt rows, clusters and one block a row;
    rows from none to all of the keys the table can hold."""
    cache = filled([most], 16, 4, E4M3, seed=rows)
    rng = np.random.RandomState(rows)
    n = rng.randint(0, most + 1, rows)
    n[rng.randint(0, rows, 2)] = [0, most]
    check_attn(cache, randn(6, rows, 8, 128), n, seq=[0] * rows)


def test_graph_of_dealt_rows_and_two_calls_at_once(cuda_ok):
    """Long rows shared by blocks and joined by a second kernel: captured and replayed for other lengths (none at
    all among them), and called on two streams at once with a workspace each."""
    cache = filled([9000, 5000, 20], 64, 2, INT8)
    q = randn(0, 3, 16, 128).cuda()
    out, lse = torch.full_like(q, 7.0), torch.zeros((3, 16), device="cuda")
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(dsa.workspace_size(dsa.DSA_OP_PAGED_ATTN, 1, 3, 16, 1, 1), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_paged_attn(q, cache.k, cache.v, cache.ks, cache.vs, cache.table_gpu, n, 0.1, out, lse=lse, ws=ws)
    lengths = [[9000, 5000, 20], [0, 0, 0], [1, 0, 17], [8999, 1, 0], [0, 4999, 20]]
    wants = [attend(cache, q, v, 0.1) for v in lengths]
    for v, (want, wlse) in zip(lengths, wants):
        n.copy_(torch.tensor(v, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert not wants[1][0].any() and torch.isinf(wants[1][1]).all()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for i in range(10):
        for s, (one, many) in enumerate(((0, 3), (3, 0))):
            with torch.cuda.stream(streams[s]):
                got[s].append((one, attend(cache, q, lengths[one], 0.1)))
                got[s].append((many, attend(cache, q, lengths[many], 0.1)))
    torch.cuda.synchronize()
    for which, (o, l) in got[0] + got[1]:
        assert torch.equal(o, wants[which][0]) and torch.equal(l, wants[which][1])
    ok()
