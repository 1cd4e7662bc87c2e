"""Every kernel of the product and of the quantisation, at sizes that reach it and make it go on
from one piece of work to the next, against the 64-bit forms (operator_oracles)."""
import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import operator_oracles as oo
from tests.test_gpu_operators import DT, _f64, _near, _product, _quantize

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


# Every way of the product: tiles of 16, 32, 64 and 128 tokens, undivided and with k shared by
# each number of CTAs that is chosen on a GPU of 152 SMs, with rows of y on 32 bytes, on 16 and
# off them, features and values of k that end inside a tile, and each type.
DENSE = [
    (16, 1, 1, 100, 100, "bf16", 0), (16, 2, 1, 7007, 1000, "fp32", 1), (16, 3, 9, 5001, 1000, "fp16", 7),
    (16, 4, 13, 100, 1000, "fp16", 4), (16, 5, 16, 3333, 3000, "bf16", 0), (16, 6, 1, 2007, 2000, "fp32", 0),
    (16, 8, 5, 100, 2000, "bf16", 12),
    (32, 1, 20, 100, 100, "fp32", 4), (32, 2, 20, 7007, 2000, "bf16", 1), (32, 3, 31, 5001, 2000, "fp16", 0),
    (32, 4, 20, 100, 1000, "bf16", 0), (32, 5, 17, 3333, 3000, "fp32", 3), (32, 6, 20, 2007, 2000, "fp16", 9),
    (32, 8, 20, 100, 2000, "fp32", 0),
    (64, 1, 40, 100, 100, "fp16", 12), (64, 2, 40, 7007, 1000, "fp32", 0), (64, 3, 64, 5001, 1000, "bf16", 7),
    (64, 4, 40, 100, 1000, "bf16", 0), (64, 5, 130, 1001, 3000, "fp16", 0), (64, 6, 40, 2007, 2000, "fp32", 1),
    (64, 8, 40, 100, 2000, "bf16", 4),
    (128, 1, 513, 5001, 2000, "bf16", 7), (128, 1, 700, 5001, 2000, "fp32", 7), (128, 2, 130, 7007, 2000, "bf16", 1),
    (128, 3, 130, 5001, 3000, "fp32", 0), (128, 4, 130, 3333, 2000, "fp16", 3), (128, 4, 130, 3333, 2000, "bf16", 0),
    (128, 5, 40, 7007, 4090, "fp32", 1), (128, 6, 1030, 300, 3000, "bf16", 4), (128, 6, 1030, 300, 3000, "fp32", 4),
    (128, 8, 100, 3333, 3000, "fp16", 0), (128, 8, 128, 3333, 3000, "bf16", 11),
]
# (experts, tokens of one on average); 800 and 4096 experts leave the large tiles two stages
EXPERTS = [
    (16, 4, 3, 1, 100, 1000, "bf16", 0), (16, 6, 16, 1, 100, 2000, "fp32", 0), (16, 1, 800, 1, 100, 100, "bf16", 4),
    (16, 1, 4096, 1, 70, 300, "fp32", 0), (32, 8, 3, 5, 100, 2000, "bf16", 0), (32, 1, 800, 5, 100, 100, "fp16", 0),
    (64, 3, 16, 20, 200, 1000, "fp32", 1), (64, 1, 800, 20, 100, 100, "bf16", 1), (64, 6, 16, 20, 100, 2000, "fp16", 0),
    (128, 1, 64, 128, 200, 1000, "bf16", 8), (128, 1, 64, 128, 200, 2000, "fp32", 1),
    (128, 1, 800, 20, 200, 1000, "bf16", 8), (128, 2, 64, 64, 200, 2000, "fp16", 0),
    (128, 4, 16, 128, 200, 2000, "fp32", 3), (128, 6, 16, 20, 500, 4090, "bf16", 0),
]


def _path(t, n, k, dtype, pad, experts=0):
    offsets = 0x10000 if experts else None
    return rs.reshard_fp8_matmul_path(0x10000, (t, n, k), dtype, offsets=offsets,
                                      nexperts=max(1, experts), ldy=n + pad)


def _is_path(found, tile, split):
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert found == (tile, split)


@pytest.mark.parametrize("tile,split,t,n,k,dtype,pad", DENSE)
def test_matmul_on_every_path(tile, split, t, n, k, dtype, pad):
    _is_path(_path(t, n, k, dtype, pad), tile, split)
    _near(*_product(t, n, k, dtype, seed=t + n + k, pad=pad))


@pytest.mark.parametrize("tile,split,experts,each,n,k,dtype,pad", EXPERTS)
def test_matmul_of_experts_on_every_path(tile, split, experts, each, n, k, dtype, pad):
    """Uneven experts, some without rows; rows before and after every expert's."""
    g = torch.Generator().manual_seed(experts + n)
    t = experts * each
    popular = torch.rand(experts, generator=g) ** 2 * (torch.rand(experts, generator=g) < 0.8) + 1e-6
    counts = torch.bincount(torch.multinomial(popular, t - 2, replacement=True, generator=g), minlength=experts)
    _is_path(_path(t, n, k, dtype, pad, experts), tile, split)
    _near(*_product(t, n, k, dtype, experts, counts.tolist(), seed=n + k, pad=pad, rows=1))


def test_matmul_path_of_nothing_and_refusals():
    for shape in ((0, 5, 5), (5, 0, 5), (5, 5, 0)):
        assert _path(*shape, "bf16", 0) == (0, 0)
    for kw in (dict(ldy=4), dict(nexperts=2), dict(offsets=3)):
        with pytest.raises(rs.ReshardError):
            rs.reshard_fp8_matmul_path(0x10000, (5, 5, 128), "bf16", **kw)
    with pytest.raises(rs.ReshardError):
        rs.reshard_fp8_matmul_path(None, (5, 5, 128), "bf16")


# --------------------------------------------------------------------------- quantize
@pytest.mark.parametrize("rows,cols,ldx,ldq,shift,dtype", [
    (5001, 2048, None, None, 0, "bf16"),   # several rows a lane, whole vectors
    (40003, 300, 304, 304, 8, "fp16"),     # ragged width, rows on 16 bytes
    (33001, 259, None, None, 1, "bf16"),   # off them
    (66000, 100, 101, 103, 1, "fp32"),
])
def test_quantize_of_many_rows(rows, cols, ldx, ldq, shift, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(1, rows, cols, generator=g, device="cuda") * 3).to(DT[dtype])
    q, s = _quantize(x, 1, ldx, ldq, None, shift, dtype)
    wq, ws = oo.quantize(_f64(x), 1)
    assert np.array_equal(s, ws) and np.array_equal(q, wq)
