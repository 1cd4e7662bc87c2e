"""Gradients of the scores at temperatures next to 0 on a GB300: 1 / T near float32's largest number, where
products with it leave the range, against the plain 64-bit form (logit_oracles)."""
import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import logit_oracles as lo
from tests.test_gpu_logprob import DT, EPS, _f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(8, 700), (8, 40001)])
@pytest.mark.parametrize("g,h", [(0.25, -0.5), (0.0, 1.0), (-0.5, 0.25), (0.5, 0.0)])
def test_gradient_next_to_temperature_0(g, h, rows, vocab, dtype):
    """Differences of logits are 2^-8 at least or 0: beside the largest ones every probability is 0, and with
    |g| and |h| of at most 1 / 2 and 1 no gradient leaves float32's range."""
    x = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(vocab)).mul(256).round().div(256)
    x[:, 11] = 7.0
    x[3, 12] = x[5, 600] = 7.0              # two that share all
    x = x.to(DT[dtype])
    t = torch.tensor([1e-35, 1e-36, 3e-37, 1e-37, 2e-38, 1.2e-38, 1e-39, 1e-45])
    target = torch.tensor([11, 4, 11, 12, 5, 11, 600, 11], dtype=torch.int32)
    state, grad = torch.empty(rows, 4, device="cuda"), torch.empty_like(x, device="cuda")
    kw = dict(target=target.cuda(), temperature=t.cuda())
    rs.reshard_logprob(x.cuda(), (rows, vocab), dtype, state=state, **kw)
    rs.reshard_logprob_grad(x.cuda(), (rows, vocab), dtype, state, grad, dlogprob=torch.full((rows,), g, device="cuda"),
                            dentropy=torch.full((rows,), h, device="cuda"), **kw)
    torch.cuda.synchronize()
    got = _f64(grad)
    for r in range(rows):
        want, bound = lo.logprob_grad(lo.cleaned(_f64(x[r]), dtype), float(t[r]), int(target[r]), g, h, EPS[dtype])
        assert np.all(np.isfinite(got[r])), (r, np.flatnonzero(~np.isfinite(got[r]))[:5])
        assert np.all(np.abs(got[r] - want) <= bound), (r, np.max(np.abs(got[r] - want) - bound))
