"""Argument checks of distillation, without a GPU: every refusal comes before any device work, with a
message, and calls with nothing to do are accepted; and the oracle's gradient against differences of
its loss."""
import numpy as np
import pytest

import dtensor_reshard_gb300 as rs
from tests import logit_oracles as lo

P, Q = 0x10000, 0x20000     # addresses that are never dereferenced
INVALID, UNSUPPORTED = 1, 2


def _refused(status, call, *args, **kw):
    with pytest.raises(rs.ReshardError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    assert rs.reshard_last_error()


def test_distill_refusals():
    def call(logits=P, shape=(2, 50), dtype="bf16", token=P, y=P, ntop=4, loss=Q, dlogits=Q, **kw):
        rs.reshard_distill_loss(logits, shape, dtype, token, y, ntop, loss=loss, dlogits=dlogits, **kw)
    for kw in (dict(logits=None), dict(token=None), dict(y=None), dict(dtype="i64"), dict(shape=(-2, 50)),
               dict(shape=(2, -50)), dict(ntop=0), dict(ntop=-1), dict(ld=49), dict(ldtop=3), dict(logits=P + 1),
               dict(dlogits=Q + 1), dict(token=P + 2), dict(y=P + 1), dict(loss=Q + 2), dict(grad=P + 1),
               dict(temperature=P + 3)):
        _refused(INVALID, call, **kw)
    for kw in (dict(shape=(2, rs.MAX_VOCAB + 1)), dict(shape=(1 << 28, 50)), dict(shape=(1 << 62, 50)),
               dict(ntop=rs.MAX_TOP + 1)):
        _refused(UNSUPPORTED, call, **kw)
    call(None, (0, 50), token=None, y=None, loss=None, dlogits=None)
    call(None, (2, 0), token=None, y=None, loss=None, dlogits=None)
    call(loss=None, dlogits=None)                        # nothing asked for


@pytest.mark.parametrize("tail", [False, True])
def test_the_oracles_gradient(tail):
    g = np.random.default_rng(3)
    x, token, y = g.normal(size=30), np.array([3, 9, 3, 29, -1]), np.log(np.array([0.3, 0.2, 0.1, 0.15, 0.1]))
    loss = lambda a: lo.distill(a, 0.7, token, y, tail, 1.0, (0.0, 0.0))[0]  # noqa: E731
    grad = lo.distill(x, 0.7, token, y, tail, 1.0, (0.0, 0.0))[2]
    for i in range(30):
        step = np.zeros(30)
        step[i] = 1e-5
        assert abs((loss(x + step) - loss(x - step)) / 2e-5 - grad[i]) < 1e-8


def test_the_oracles_gradient_of_scores():
    g = np.random.default_rng(4)
    x = g.normal(size=30)
    value = lambda a: 1.3 * lo.logprob(a, 0.7, 5)[0] - 0.4 * lo.entropy(a, 0.7)[0]  # noqa: E731
    grad = lo.logprob_grad(x, 0.7, 5, 1.3, -0.4, (0.0, 0.0))[0]
    for i in range(30):
        step = np.zeros(30)
        step[i] = 1e-5
        assert abs((value(x + step) - value(x - step)) / 2e-5 - grad[i]) < 1e-8
