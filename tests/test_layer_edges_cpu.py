"""Edges of the layer operators' host side: statuses, refusals, empty calls, builds."""
import ctypes

import pytest
import torch

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


def test_rows_of_empty_tensors(lib):
    """Any layout of no rows is one stride; what has rows is checked as before."""
    e, z = torch.empty, torch.zeros
    assert gdn._rows("q", e(2, 0, 3, 64), 2) == 192
    assert gdn._rows("q", e(0, 5, 3, 64), 2) == 192
    assert gdn._rows("g", e(3, 0, 4), 1) == 4
    assert gdn._rows("q", z(4, 8, 16)[:2, :0, 8:], 1) == 8
    with pytest.raises(ValueError):
        gdn._rows("q", z(4, 8, 16)[:2, :1, ::2], 1)
    with pytest.raises(ValueError):
        gdn._rows("q", z(4, 8, 16)[:2, :3], 1)
