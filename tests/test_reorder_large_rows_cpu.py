"""A state that the reordering cannot take is refused before any other state of the call is
touched, wherever it stands in the list."""
import ctypes
import struct

import pytest
import torch

from test_abi import _load

PASSED = (-7, -8)  # what a valid call comes to without a GPU


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("argument checks with made-up device pointers run only without a GPU")
    return _load()


@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("before", [0, 1, 20, 700])
def test_rows_of_too_many_vectors(lib, place, before):
    def state(i, size, stride, segments=1, seg=0):
        at = (i + 1) << 44
        return struct.pack("<QQqqqqqq", at, at if place else at + (1 << 43), stride, stride, segments,
                           seg or size, seg or size, size)

    def call(*big):
        small = b"".join(state(i, 64, 64) for i in range(before))
        last = state(before, *big)
        return lib.pstat_beam_reorder(small + last, before + 1, ctypes.c_void_p(0x9000000), 2, 4, 4, None,
                                      None)
    most = (1 << 32) - 257
    assert call(most, most) in PASSED  # bytes
    assert call(most + 2, most + 2) == -2
    assert call(16 * most, 16 * most) in PASSED  # the same in vectors of 16
    assert call(16 * most + 16, 16 * most + 16) == -2
    assert call(3, 1 << 36, 1 << 31, 7) == -2  # runs
    assert call(3, 1 << 36, 1 << 30, 7) in PASSED
