"""The 8-bit path's limits and modules without a GPU."""
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb

OK, INVALID = 0, 1
BF16 = 2


@pytest.mark.parametrize("M, K, within", [
    ((1 << 28) - 16, 16, True), ((1 << 28) - 15, 16, False), ((1 << 28) - 1, 128, False),
    ((1 << 27) - 8, 144, True), ((1 << 27) - 7, 144, False), ((1 << 12) - 1, 1 << 23, True), (1 << 12, 1 << 23, False),
])
def test_quantize_act_f8_takes_no_more_than_a_launch_can_hold(lowbit_lib, M, K, within):
    """16 threads a block of 128: 2^32 - 256 threads at most.  (The sizes are checked before the
    NULL pointers.)"""
    assert lowbit_lib.lowbit_quantize_act_f8(None, BF16, M, K, None, None, None) == INVALID
    assert ("NULL" in lb.lowbit_last_error()) == within
    assert ("2^28 - 16" in lb.lowbit_last_error()) != within
