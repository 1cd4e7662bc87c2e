"""The operators' kernels at sizes that make them go on from one piece of work to the next,
against the 64-bit forms (operator_oracles)."""
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests.test_gpu_operators import _near, _product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    yield
    assert rs.reshard_device_status(clear=True) == 0


# pad: of y's rows, in elements
@pytest.mark.parametrize("t,n,k,dtype,pad", [
    (2100, 5120, 1024, "bf16", 0),    # rows of y on 32 bytes, short last tiles of tokens
    (2100, 5001, 1000, "fp16", 7),    # and of features, and a short last block of k
    (2100, 5000, 4096, "bf16", 0),    # rows of y on 16 bytes
    (2100, 5001, 4096, "fp32", 0),    # on 4
    (2500, 8200, 2500, "fp32", 3),
])
def test_matmul_of_several_tiles_a_cta(t, n, k, dtype, pad):
    """More tiles of 128 tokens x 256 features than SMs."""
    _near(*_product(t, n, k, dtype, seed=t + n + k, pad=pad))


@pytest.mark.parametrize("counts,n,k,dtype,pad", [
    ([700, 0, 129, 1500, 1, 2300, 128, 0], 3000, 1024, "bf16", 8),
    ([1, 0, 0, 4000, 900, 33], 2050, 4000, "fp32", 0),
])
def test_matmul_of_experts_of_several_tiles_a_cta(counts, n, k, dtype, pad):
    _near(*_product(sum(counts) + 9, n, k, dtype, len(counts), counts, seed=n, pad=pad, rows=4))
