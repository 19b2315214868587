"""How the Python binding turns its arguments into addresses (no GPU)."""
import enum
import sys

import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq


class Place(enum.IntEnum):
    A = 4096


class Rows(np.ndarray):
    pass


HOST = np.arange(8)
TENSOR = torch.arange(8)


@pytest.mark.parametrize("arg,want", [(None, None), (0, 0), (1 << 40, 1 << 40), (Place.A, 4096), (HOST, HOST.ctypes.data), (HOST[2:], HOST.ctypes.data + 16),
                                      (HOST.view(Rows), HOST.ctypes.data), (TENSOR, TENSOR.data_ptr()), (TENSOR[3:], TENSOR.data_ptr() + 24)])
def test_addresses(arg, want):
    assert hq._dp(arg) == want


@pytest.mark.parametrize("arg", [None, 1 << 20, HOST, TENSOR])
def test_plain_arguments_raise_nothing_on_the_way(arg):
    """An exception caught on the way costs 0.3 us an address: calls with plain addresses took 2 us more."""
    raised = []

    def trace(frame, event, _):
        if event == "exception":
            raised.append(frame.f_code.co_name)
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        hq._dp(arg)
    finally:
        sys.settrace(before)
    assert not raised


def test_what_has_no_address_is_refused():
    for arg in ("x", 1.5, [1, 2]):
        with pytest.raises(AttributeError):
            hq._dp(arg)
