"""Edges of the layer operators' host side: statuses, refusals, empty calls, builds."""
import ctypes

import pytest

from chunked_linear_recurrence_gated_gb300 import build, gdn

P = ctypes.c_void_p
FAKE = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def test_exchange_check_refuses_bad_arguments(lib):
    for sums, silent in ((None, -1), (FAKE + 2, -1), (FAKE, -2), (FAKE, 4)):
        assert lib.gdn_diag_exchange(P(sums) if sums else None, silent, 20, None) == 1
