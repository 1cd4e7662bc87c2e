"""What the binding takes for an address, without a GPU."""
import ctypes

import numpy as np
import pytest

import dtensor_reshard_gb300 as rs


class _Buffer:
    """An object that says where its data lies, by a number that is no Python int."""

    def __init__(self, at):
        self.at = at

    def data_ptr(self):
        return self.at


@pytest.mark.parametrize("address", [0x10000, np.int64(0x10000), np.uint64(0x10000)])
def test_addresses(address):
    for x in (address, _Buffer(address)):
        got = rs._ptr(x)
        assert type(got) is int and got == 0x10000
        assert ctypes.c_void_p(got).value == 0x10000
        rs.reshard_expert_dispatch(x, (0, 2, 128), "bf16", x, x)        # nothing to do, but an address in each place


def test_no_address():
    for x in (None, 0, np.int64(0), _Buffer(0), _Buffer(np.int64(0))):
        assert rs._ptr(x) is None
