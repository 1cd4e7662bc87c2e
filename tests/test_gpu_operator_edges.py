"""Values and sizes at the ends of the operators' ranges, against the 64-bit forms."""
import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import operator_oracles as oo
from tests.test_gpu_operators import DT, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    yield
    assert rs.reshard_device_status(clear=True) == 0


# --------------------------------------------------------------------------- quantize
def _bytes(values, negative):
    """The e4m3 bytes of values with the given signs (of zeros too)."""
    table = oo.e4m3_values()[:127]
    return np.searchsorted(table, np.abs(values)).astype(np.uint8) | (negative.astype(np.uint8) << 7)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [256, 203])
def test_quantize_keeps_the_sign_of_zeros(cols, dtype, block_rows):
    """x / scale is -0 where x is, and rounds to -0 where x is small and negative."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(150, cols, generator=g, device="cuda")
    x[:, ::3] = -0.0
    x[:, 1::9] = 0.0
    x[:, 2::9] *= 1e-4
    x[5] = -0.0                              # (blocks of zeros alone)
    if dtype == "fp32":
        x[130:] *= 1e-32                     # (scales below 2^-90)
    x = x.to(DT[dtype])
    q = torch.empty(150, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-150 // block_rows), -(-cols // 128), device="cuda")
    rs.reshard_fp8_quantize(x, q, s, (150, cols), dtype, block_rows)
    want, _ = oo.quantize(_f64(x)[None], block_rows)
    negative = torch.signbit(x).cpu().numpy()
    assert np.array_equal(q.cpu().numpy(), _bytes(want[0], negative))
