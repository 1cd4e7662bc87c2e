"""Distillation where the loss reaches the end of float32's range on a GB300: a student that is sure of a token
of which its teacher knows nothing, by a logit of +inf or of the type's largest value."""
import math

import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import logit_oracles as lo
from tests.test_gpu_distill import DT, EPS, _f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("k", [1, 4, 33, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_a_loss_at_the_end_of_the_range(dtype, k, tail):
    """Float32's largest number times probabilities that add up to 1 within a rounding or so: that number within
    the oracle's bound, or +inf where the bound reaches beyond it."""
    rows, vocab = 24, 700
    g = torch.Generator().manual_seed(k)
    x = torch.randn(rows, vocab, generator=g)
    x[:, 5] = math.inf
    x[1::2, 5] = lo.LARGEST[dtype]
    token = torch.stack([6 + torch.randperm(vocab - 6, generator=g)[:k] for _ in range(rows)]).to(torch.int32)
    y = torch.log_softmax(torch.randn(rows, k, generator=g), 1)
    if tail:
        y[::3] += 2.0                       # a list whose probabilities are beyond 1
    x = x.to(DT[dtype])
    loss, grad = torch.empty(rows, device="cuda"), torch.empty(rows, vocab, dtype=DT[dtype], device="cuda")
    rs.reshard_distill_loss(x.cuda(), (rows, vocab), dtype, token.cuda(), y.cuda(), k, loss=loss, dlogits=grad, tail=tail)
    torch.cuda.synchronize()
    top = float(np.finfo(np.float32).max)
    for r in range(rows):
        want, bound, dl, off = lo.distill(lo.cleaned(_f64(x[r]), dtype), 1.0, token[r].numpy(), _f64(y[r]), tail, 1.0, EPS[dtype])
        got = float(loss[r])
        assert abs(got - want) <= bound or (got == math.inf and want + bound >= top), (r, got, want, bound)
        assert np.all(np.abs(_f64(grad[r]) - dl) <= off)
