"""pstat_beam_gather's argument checks: those of pstat_beam_reorder, and no call in place."""
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


def test_gather_argument_checks(lib):
    plain = (0x1000000, 0x2000000, 64, 64, 1, 64, 64, 64)

    def call(*states, parents=0x9000000, B=2, beams=3, out_beams=3):
        b = b"".join(struct.pack("<QQqqqqqq", *s) for s in states)
        return lib.pstat_beam_gather(b or None, len(states), ctypes.c_void_p(parents), B, beams, out_beams,
                                     None, None)
    assert call(plain) in PASSED and call(plain, out_beams=7) in PASSED and call() == 0
    assert call(plain, parents=0) == -1 and call(plain, parents=0x9000004) == -5
    assert call(plain, beams=65) == -2 and call(plain, out_beams=0) == -2
    here = (0x1000000, 0x1000000, 64, 64, 1, 64, 64, 64)
    assert call(here) == -9
    assert call((0x1000000, 0x1000020) + plain[2:]) == -9


def test_native_binding_refuses_no_address():
    from test_binding_cpu import native

    for args in ((), (0,), (1, 2)):
        with pytest.raises(ValueError):
            native.bind_gather(*args)
