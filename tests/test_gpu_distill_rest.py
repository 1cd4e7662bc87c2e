"""Distillation with the teacher's rest where the student is sure of its listed tokens: loss and gradient
on a GB300 against a 64-bit form that works with logarithms (rest_oracles)."""
import math

import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import logit_oracles as lo
from tests import rest_oracles as ro
from tests.test_gpu_distill import DT, EPS, _f64, _placed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    yield
    assert rs.reshard_device_status(clear=True) == 0


def _case(rows, vocab, k, gap, t, rest, seed):
    """Listed tokens about gap * t above the others, a teacher whose list has 1 - rest."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * 3 * t
    token = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(rows)]).to(torch.int32)
    x.scatter_(1, token.long(), (gap + torch.rand(rows, k, generator=g) * 4) * t)
    share = torch.softmax(torch.randn(rows, k, generator=g, dtype=torch.float64), 1) * (1 - rest)
    return x, token, share.log().float(), torch.rand(rows, generator=g) + 0.5


def _check(x, dtype, token, y, t, grad, shift=0, other=0, inplace=False, rows=None):
    n, vocab = x.shape
    k, ld = token.shape[1], vocab + 3
    temperature = torch.full((n,), t)
    buf, view = _placed(x.cuda(), ld, shift, 50.0)
    out, oview = (buf, view) if inplace else _placed(torch.full_like(x, 9.0).cuda(), ld, other, 50.0)
    loss = torch.full((n,), 7.0, device="cuda")
    rs.reshard_distill_loss(buf, (n, vocab), dtype, token.cuda(), y.cuda(), k, loss=loss, dlogits=out, tail=True,
                            temperature=temperature.cuda(), grad=grad.cuda(), ld=ld)
    torch.cuda.synchronize()
    assert bool((oview[:, vocab:] == 50.0).all())
    got = _f64(oview[:, :vocab])
    for r in range(n) if rows is None else rows:
        l, lb, want, bound = ro.distill(lo.cleaned(_f64(x[r]), dtype), float(temperature[r]), token[r].numpy(), _f64(y[r]),
                                        float(grad[r]), EPS[dtype])
        assert abs(float(loss[r]) - l) <= lb, (r, float(loss[r]), l, lb)
        assert np.all(np.abs(got[r] - want) <= bound), (r, np.max(np.abs(got[r] - want) / bound))
        assert float(loss[r]) >= -lb
        assert abs(got[r].sum() - want.sum()) <= bound.sum()
    return loss


@pytest.mark.parametrize("t", [1.0, 0.1, 0.01])
@pytest.mark.parametrize("gap", [20, 80, 88, 100, 300, 740, 2000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 131072, 64), (3, 50021, 5), (200, 4099, 20), (6, 129, 128)])
def test_a_student_that_is_sure(rows, vocab, k, dtype, gap, t):
    x, token, y, grad = _case(rows, vocab, k, gap, t, 0.1, rows + gap)
    x = x.to(DT[dtype])
    pick = range(0, rows, max(1, rows // 3))
    _check(x, dtype, token, y, t, grad, rows=pick)
    _check(x, dtype, token, y, t, grad, shift=1, other=2, rows=pick)
    _check(x, dtype, token, y, t, grad, shift=3, inplace=True, rows=pick)


@pytest.mark.parametrize("rest", [2.0 ** -20, 2.0 ** -10, 0.05, 0.5, 0.9])
@pytest.mark.parametrize("gap", [60, 87, 90, 500])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rests_of_every_size(dtype, gap, rest):
    x, token, y, grad = _case(5, 3001, 33, gap, 0.5, rest, gap)
    _check(x.to(DT[dtype]), dtype, token, y, 0.5, grad)


def test_one_listed_token_and_a_jump_that_is_not_there():
    """One token with probability 0.9, all others a little further below it at T = 0.1 from case to case: the
    loss grows by 0.1 times the gap over T and nothing else."""
    vocab = 131072
    token, y = torch.zeros(1, 1, dtype=torch.int32), torch.tensor([[math.log(0.9)]])
    losses = []
    for gap in (8.0, 8.5, 8.75, 9.0, 9.5, 10.5, 12.0):
        x = torch.zeros(1, vocab)
        x[0, 0] = gap
        losses.append((gap, float(_check(x, "fp32", token, y, 0.1, torch.ones(1)))))
    for (a, la), (b, lb) in zip(losses, losses[1:]):
        assert abs((lb - la) - 0.1 * (b - a) / 0.1) < 1e-4       # gaps are exact, losses below 16


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_masks_and_tokens_of_the_row_s_ends(dtype):
    n, vocab, k = 6, 1000, 8
    x, token, y, grad = _case(n, vocab, k, 95, 1.0, 0.2, 7)
    token[0] = torch.tensor([0, 1, 2, 3, vocab - 1, vocab - 2, vocab - 3, vocab - 4])
    x[0] = -3.0
    x[0, token[0].long()] = 95.0
    off = torch.ones(vocab, dtype=torch.bool)
    for r, low in ((1, -math.inf), (2, -lo.LARGEST[dtype]), (3, -1e4), (4, math.nan)):
        off[:] = True
        off[token[r].long()] = False
        off[500] = r > 2                  # (in rows 1 and 2 one token is left for the rest)
        x[r, off] = low
    x[5, 17] = -math.inf
    token[5, 3], token[5, 4] = token[5, 0], -1
    _check(x.to(DT[dtype]), dtype, token, y, 1.0, grad)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_everything_else_masked(dtype):
    """Nothing outside the list but what is masked, by -inf or the type's lowest value: the rest has nowhere to be."""
    x, token, y, grad = _case(2, 900, 6, 4, 1.0, 0.2, 9)
    for r, low in ((0, -math.inf), (1, -lo.LARGEST[dtype])):
        keep = x[r, token[r].long()].clone()
        x[r] = low
        x[r, token[r].long()] = keep
    _check(x.to(DT[dtype]), dtype, token, y, 1.0, grad)
