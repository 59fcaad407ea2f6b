"""The frequencies of rope_freqs against the published formulas, pair by pair (host only)."""
import math

import numpy as np
import pytest

import dsa_lightning_indexer_02_b200 as dsa


def yarn(rot, theta, factor, orig_len, fast=32.0, slow=1.0):
    """YaRN's mix: pair index d(b) turns b times over orig_len positions; the ramp runs from floor(d(fast)), at least 0,
    to ceil(d(slow)), at most rot - 1.  Where the first passes the second, every pair turns more than `fast` times."""
    f = theta ** (-np.arange(rot // 2) / (rot / 2))
    d = lambda b: rot * math.log(orig_len / (b * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(d(fast)), 0), min(math.ceil(d(slow)), rot - 1)
    r = np.clip((np.arange(rot // 2) - lo) / (hi - lo), 0, 1) if hi > lo else np.arange(rot // 2) > lo
    return f * (1 - r) + f / factor * r, f


SETTINGS = [
    (64, 1e4, 8.0, 4096), (128, 1e6, 4.0, 32768),                        # the ramp ends among the pairs
    (64, 1e4, 8.0, 131072), (128, 1e4, 4.0, 131072), (64, 1e4, 8.0, 65536), (32, 5e3, 32.0, 50000),   # behind the last one
    (16, 1e4, 32.0, 1 << 20), (16, 1e4, 2.0, 1 << 40), (2, 1e4, 4.0, 4096), (256, 1e4, 1.0, 4096),
]


@pytest.mark.parametrize("rot,theta,factor,orig_len", SETTINGS)
def test_yarn_is_the_published_mix(rot, theta, factor, orig_len):
    got, m = dsa.rope_freqs(rot, theta, "yarn", factor, orig_len)
    want, plain = yarn(rot, theta, factor, orig_len)
    assert np.allclose(got.numpy(), want, rtol=1e-12, atol=0)
    assert math.isclose(m, 0.1 * math.log(factor) + 1 if factor > 1 else 1.0, rel_tol=1e-6)
    turns = orig_len * plain / (2 * math.pi)
    ratio = got.numpy() / plain
    assert np.allclose(ratio[turns > 32.0], 1.0, rtol=1e-12)
    assert np.allclose(ratio[turns < 1.0], 1 / factor, rtol=1e-12)
    assert factor == 1.0 or np.all(ratio[turns > 1.0 + 1e-9] > 1 / factor * (1 + 1e-9)) or turns.min() > 32


@pytest.mark.parametrize("fast,slow", [(16.0, 2.0), (64.0, 0.5)])
def test_yarn_with_other_bounds(fast, slow):
    got, _ = dsa.rope_freqs(64, 1e4, "yarn", 8.0, 65536, fast, slow)
    assert np.allclose(got.numpy(), yarn(64, 1e4, 8.0, 65536, fast, slow)[0], rtol=1e-12, atol=0)
