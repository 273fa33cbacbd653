"""Rotary outputs that start where the other output or the other input does: each is
read and written by blocks of its own, in no order, so the call is refused (CPU; the
pointers are never dereferenced)."""
import ctypes

import pytest

from gated_delta_rule_60_b200 import binding, build

P = ctypes.c_void_p
INV = binding.KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("q,k,qo,ko", [(1024, 2048, 4096, 4096), (1024, 2048, 2048, 4096), (1024, 2048, 4096, 1024),
                                       (1024, 2048, 2048, 1024)])
def test_overlap_is_refused(q, k, qo, ko):
    build.build()
    lib = binding.load_library()
    for Hq, Hk in ((2, 2), (4, 2)):
        assert lib.kda_rotary(P(q), P(k), P(256), P(256), None, 1, 4, Hq, Hk, 64, 64, 0, 0, 0, 1.0, Hq * 64, Hk * 64,
                              P(qo), P(ko), Hq * 64, Hk * 64, None) == INV
