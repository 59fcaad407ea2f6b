"""Keys whose rotation comes out next to a chosen value: for tests of what fp32's own error could decide wrongly."""
from __future__ import annotations

import numpy as np


def bf16(x):
    """The nearest bf16 values, as float64 (ties away from zero: any neighbour will do here)."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32)
    return ((b + 0x8000) & np.uint32(0xffff0000)).view(np.float32).astype(np.float64)


def turned(pos, a, b):
    """(a cos pos - b sin pos, a sin pos + b cos pos) with the angle in extended precision."""
    ang = np.asarray(pos, dtype=np.longdouble)
    c, s = np.cos(ang), np.sin(ang)
    return a * c - b * s, a * s + b * c


def near(targets, seed, count, within=2.0 ** -23, beyond=2.0 ** -33, most=20000):
    """`count` rows (pos, a, b, target), 0 < pos < most, a and b in bf16, with a cos pos - b sin pos within the given
    relative distance of one of the targets, but no nearer than `beyond` of |a| + |b|: a is solved for and rounded to
    bf16, which comes that near by chance."""
    rng = np.random.RandomState(seed)
    got = []
    while sum(len(g) for g in got) < count:
        n = 1 << 20
        pos, t = rng.randint(1, most, n), rng.choice(targets, n)
        b = bf16(rng.uniform(-1, 1, n) * np.abs(t))
        c, s = np.cos(pos.astype(np.float64)), np.sin(pos.astype(np.float64))
        with np.errstate(divide="ignore", invalid="ignore"):
            a = bf16(np.where(np.abs(c) > 0.3, (t + b * s) / c, 0))
        some = np.flatnonzero(np.abs(a * c - b * s - t) <= 2 * within * np.abs(t))
        pos, a, b, t = pos[some], a[some], b[some], t[some]
        y, z = turned(pos, a, b)
        far = np.abs(y - t)
        ok = (far <= within * np.abs(t)) & (far >= beyond * (np.abs(a) + np.abs(b))) & (np.abs(z) < 0.98 * np.abs(t))
        got.append(np.stack([pos[ok], a[ok], b[ok], t[ok]], 1))
    return np.concatenate(got)[:count]
