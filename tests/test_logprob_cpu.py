"""Argument checks of scores of logits and their gradient, without a GPU: every refusal comes before
any device work, with a message, and calls with nothing to do are accepted."""
import pytest

import dtensor_reshard_gb300 as rs

P, Q = 0x10000, 0x20000     # addresses that are never dereferenced
INVALID, UNSUPPORTED = 1, 2


def _refused(status, call, *args, **kw):
    with pytest.raises(rs.ReshardError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    assert rs.reshard_last_error()


def test_logprob_refusals():
    def call(logits=P, shape=(2, 50), dtype="bf16", target=P, logprob=Q, **kw):
        rs.reshard_logprob(logits, shape, dtype, target=target, logprob=logprob, **kw)
    top = dict(top_token=Q, top_logprob=Q, ntop=3)
    for kw in (dict(logits=None), dict(target=None), dict(dtype="i64"), dict(shape=(-2, 50)), dict(shape=(2, -50)),
               dict(ld=49), dict(logits=P + 1), dict(target=P + 2), dict(logprob=Q + 1), dict(entropy=Q + 2),
               dict(temperature=P + 1), dict(state=Q + 8), dict(ntop=-1), dict(top, ldtop=2),
               dict(top, top_token=None), dict(top, top_logprob=None), dict(top, top_token=Q + 1),
               dict(top, top_logprob=Q + 2)):
        _refused(INVALID, call, **kw)
    for kw in (dict(shape=(2, rs.MAX_VOCAB + 1)), dict(shape=(1 << 28, 50)), dict(shape=(1 << 62, 50)),
               dict(top, ntop=rs.MAX_TOP + 1)):
        _refused(UNSUPPORTED, call, **kw)
    call(None, (0, 50), target=None, logprob=None)
    call(None, (2, 0), target=None, logprob=None)
    call(P, (2, 50), target=None, logprob=None)          # nothing asked for


def test_gradient_refusals():
    def call(logits=P, shape=(2, 50), dtype="bf16", state=P, dlogits=Q, target=P, dlogprob=P, **kw):
        rs.reshard_logprob_grad(logits, shape, dtype, state, dlogits, target=target, dlogprob=dlogprob, **kw)
    for kw in (dict(logits=None), dict(state=None), dict(dlogits=None), dict(target=None), dict(dtype="u8"),
               dict(shape=(-2, 50)), dict(shape=(2, -50)), dict(ld=49), dict(logits=P + 1), dict(dlogits=Q + 1),
               dict(state=P + 4), dict(target=P + 2), dict(dlogprob=P + 1), dict(dentropy=P + 2),
               dict(temperature=P + 3)):
        _refused(INVALID, call, **kw)
    for kw in (dict(shape=(2, rs.MAX_VOCAB + 1)), dict(shape=(1 << 28, 50)),
               dict(shape=((1 << 28) - 1, rs.MAX_VOCAB), ld=rs.MAX_VOCAB)):
        _refused(UNSUPPORTED, call, **kw)
    call(None, (0, 50), state=None, dlogits=None, target=None, dlogprob=None)
    call(None, (2, 0), state=None, dlogits=None, target=None, dlogprob=None)
