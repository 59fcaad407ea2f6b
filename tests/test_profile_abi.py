"""dsa_profile_end writes the eight entries that callers built against earlier headers have room for, and no more."""
import ctypes

import pytest
import torch

import dsa_lightning_indexer_02_b200 as dsa

lib = dsa.lib()
KINDS = len(dsa.PROFILE_KINDS)


def arrays(n):
    return (ctypes.c_int64 * n)(*[-7] * n), (ctypes.c_double * n)(*[-7.0] * n)


def test_profile_end_keeps_to_eight_entries():
    launches, ms = arrays(KINDS + 4)
    lib.dsa_profile_begin()
    assert lib.dsa_profile_end(launches, ms) == dsa.DSA_OK
    assert list(launches) == [0] * 8 + [-7] * (KINDS - 4) and list(ms) == [0.0] * 8 + [-7.0] * (KINDS - 4)


@pytest.mark.parametrize("n", [0, 3, KINDS, KINDS + 3])
def test_profile_end_kinds_fills_what_it_is_told(n):
    launches, ms = arrays(KINDS + 4)
    lib.dsa_profile_begin()
    assert lib.dsa_profile_end_kinds(n, launches, ms) == dsa.DSA_OK
    assert list(launches) == [0] * n + [-7] * (KINDS + 4 - n) and list(ms) == [0.0] * n + [-7.0] * (KINDS + 4 - n)
    assert lib.dsa_profile_end_kinds(-1, launches, ms) == dsa.DSA_ERR_INVALID_ARG
    lib.dsa_profile_begin()
    assert lib.dsa_profile_end_kinds(KINDS, None, None) == dsa.DSA_OK


@pytest.mark.gpu
def test_later_kinds_are_counted(cuda_ok):
    x = torch.randn(4, 2, 64, device="cuda")
    f = dsa.rope_freqs(64)[0].cuda()
    for eight in (False, True):
        dsa.profile_begin()
        dsa.dsa_rope(x, torch.empty_like(x), f)
        if eight:
            launches, ms = arrays(12)
            assert lib.dsa_profile_end(launches, ms) == dsa.DSA_OK
            assert list(launches) == [0] * 8 + [-7] * 4
        else:
            got = dsa.profile_end()
            assert got["rope"]["launches"] == 1 and got["rope"]["ms"] > 0
            assert sum(v["launches"] for v in got.values()) == 1
