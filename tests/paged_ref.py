"""The paged 8-bit cache operators in 64 bits (angles in extended precision), for the tests: plain loops over
their definitions, sharing no code with the CUDA path."""
from __future__ import annotations

import numpy as np
import torch

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
TOP = {E4M3: 448.0, INT8: 127.0}
E_MIN = -64


def rope(x, pos, inv_freq, off=0, inter=False, mscale=1.0, inverse=False):
    """(y, |a| + |b| of each element's pair, its angle's size): float64 [T, H, D]; the sizes are 0 where dims are copied."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.longdouble)
    n = len(f)
    ang = np.asarray(pos, dtype=np.longdouble)[:, None] * f
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    if inverse:
        s = -s
    one = off + (2 * np.arange(n) if inter else np.arange(n))
    two = one + (1 if inter else n)
    y, size, far = x.copy(), np.zeros_like(x), np.zeros_like(x)
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = mscale * (a * c - b * s), mscale * (a * s + b * c)
    size[..., one] = size[..., two] = abs(mscale) * (np.abs(a) + np.abs(b))
    far[..., one] = far[..., two] = np.abs(ang).astype(np.float64)[:, None]
    return y, size, far


def exponent(amax: float, fmt) -> int:
    e = E_MIN
    while amax > TOP[fmt] * 2.0 ** e:
        e += 1
    return e


def round8(x, fmt):
    """The nearest values that the format holds (ties to even, saturating): float64."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == INT8:
        return np.clip(np.rint(x), -127, 127)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)


def step8(x, fmt):
    """The distance between the format's values around x."""
    if fmt == INT8:
        return np.ones_like(x)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30)))
    return 2.0 ** (np.maximum(e, -6) - 3)


def attn(q, k_pages, v_pages, k_scale, v_scale, table, n_keys, scale, seq=None, idx=None):
    """out, lse in float64 and the tolerances of each: q bf16 [T, Hq, D] and the cache on the CPU.

    Tolerances, from the kernel's arithmetic (u = 2^-24): a logit is a sum of 128 exact products in fp32,
    off by at most 128 u A with A = scale * sum |q k| plus three roundings of its own size, so by less than
    dz = 2^-16 A; a probability is off by 2 dz and 2^-11 (its rounding to fp16; below 2^-14 by 2^-25 of the
    largest) plus 2^-20 for exponentials and fp32 sums; the output's own rounding is 2^-8.
    """
    T, Hq, D = q.shape
    page, Hkv = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    out_tol, lse_tol = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    qd = q.double().numpy()
    for t in range(T):
        n = int(n_keys[t])
        pos = np.arange(n)
        if idx is not None:
            e = np.asarray(idx[t][: min(idx.shape[1], n)])
            pos = e[(e >= 0) & (e < n)]
        if not len(pos):
            continue
        b = t if seq is None else int(seq[t])
        pid = np.asarray(table[b])[pos // page]
        k = k_pages[pid, pos % page].double().numpy() * k_scale[pid].double().numpy()[:, :, None]
        v = v_pages[pid, pos % page].double().numpy() * v_scale[pid].double().numpy()[:, :, None]
        for h in range(Hq):
            kk, vv = k[:, h // G], v[:, h // G]
            z = scale * (kk @ qd[t, h])
            dz = 2.0 ** -16 * (abs(scale) * (np.abs(kk) @ np.abs(qd[t, h]))).max()
            m = z.max()
            p = np.exp(z - m)
            l = p.sum()
            out[t, h] = (p @ vv) / l
            lse[t, h] = m + np.log(l)
            mag = (p @ np.abs(vv)) / l
            out_tol[t, h] = 2.0 ** -8 * np.abs(out[t, h]) + (2.0 ** -11 + 2.0 ** -20 + 2 * dz) * mag \
                + 2.0 ** -25 * len(pos) * (p[:, None] * np.abs(vv)).max() + 1e-38
            lse_tol[t, h] = dz + 2.0 ** -18 * (1 + abs(lse[t, h]))
    return out, lse, out_tol, lse_tol
