"""Sizes beyond what the operators' index arithmetic holds are refused before any device
work, whatever their products wrap around to."""
import pytest

import dtensor_reshard_gb300 as rs

P, Q = 0x10000, 0x20000     # addresses that are never dereferenced
UNSUPPORTED = 2


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [
    (1 << 33, 1 << 38, 64),              # nmat * row blocks wraps to 0
    ((1 << 57) + 1, 128 * 128, 64),      # to a small number
    (1, 1, (1 << 63) - 1),               # columns rounded up to blocks
    (1, (1 << 63) - 1, 1),               # rows likewise
    (1 << 31, 1, 1), (1, 1 << 38, 1), (1, 1, 1 << 38), (1 << 20, 1 << 17, 1 << 17),
])
def test_quantize_refuses_2_31_blocks_and_more(shape, block_rows):
    with pytest.raises(rs.ReshardError) as e:
        rs.reshard_fp8_quantize(P, Q, P, shape, "bf16", block_rows, lds=1 << 62)
    assert e.value.status == UNSUPPORTED, e.value


@pytest.mark.parametrize("shape", [(1 << 62, 1 << 62, 8), (1 << 31, 1, 8), (1, 1 << 31, 8), (1 << 20, 1 << 11, 8),
                                   ((1 << 63) - 1, 9, 1)])
def test_balance_workspace_of_too_many_tokens_is_none(shape):
    assert rs.reshard_balance_loss_workspace(shape) == 0


def test_balance_workspace_grows_with_the_sizes():
    sizes = [rs.reshard_balance_loss_workspace((n, t, 8)) for n, t in ((1, 1), (1, 100), (7, 100), (4000, 300),
                                                                       (1, (1 << 31) - 1))]
    assert sizes == sorted(sizes) and sizes[0] > 0
