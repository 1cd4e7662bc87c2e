"""Argument checks of the operators beside a refit, without a GPU: every refusal comes
before any device work, with a message, and calls with nothing to do are accepted."""
import numpy as np
import pytest

import dtensor_reshard_gb300 as rs
from tests import operator_oracles as oo

P, Q = 0x10000, 0x20000     # addresses that are never dereferenced


def _refused(status, call, *args, **kw):
    with pytest.raises(rs.ReshardError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    assert rs.reshard_last_error()


def test_quantize_refusals():
    def call(x=P, q=Q, s=P, shape=(2, 3, 4), dtype="bf16", **kw):
        rs.reshard_fp8_quantize(x, q, s, shape, dtype, **kw)
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(dtype="i32"), dict(dtype=99),
               dict(shape=(1, -1, 4)), dict(shape=(-1, 1, 4)), dict(shape=(1, 1, -4)),
               dict(ldx=3), dict(ldq=3), dict(lds=0), dict(block_rows=64), dict(x=P + 1), dict(s=P + 2)):
        _refused(1, call, **kw)
    for shape in ((0, 3, 4), (2, 0, 4), (2, 3, 0)):
        call(None, None, None, shape)


def test_matmul_refusals():
    def call(x=P, xs=P, w=P, ws=P, y=Q, shape=(4, 32, 64), dtype="bf16", **kw):
        rs.reshard_fp8_matmul(x, xs, w, ws, y, shape, dtype, **kw)
    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None),
               dict(dtype="u8"), dict(shape=(-1, 32, 64)), dict(shape=(4, -1, 64)),
               dict(shape=(4, 32, -1)), dict(x=P + 8), dict(w=P + 4), dict(ldx=72), dict(ldw=72),
               dict(ldx=48), dict(ldw=48), dict(ldxs=0), dict(ldws=0), dict(ldy=31), dict(xs=P + 2),
               dict(ws=P + 1), dict(y=Q + 1), dict(nexperts=3), dict(nexperts=0, offsets=P),
               dict(offsets=P + 2), dict(shape=(4, 32, 60))):
        _refused(1, call, **kw)
    _refused(2, call, nexperts=rs.MAX_EXPERTS + 1, offsets=P)
    _refused(2, call, shape=(1 << 31, 32, 64))
    _refused(2, call, shape=(4, 1 << 30, 64), nexperts=2, offsets=P)
    call(None, None, None, None, None, (0, 32, 64))
    call(None, None, None, None, None, (4, 0, 64))


def test_sample_refusals():
    def call(logits=P, shape=(2, 50), dtype="bf16", u=P, token=Q, logprob=None, **kw):
        rs.reshard_sample(logits, shape, dtype, u, token, logprob, **kw)
    for kw in (dict(logits=None), dict(u=None), dict(token=None), dict(dtype="i64"),
               dict(shape=(-2, 50)), dict(shape=(2, -50)), dict(ld=49), dict(logits=P + 1),
               dict(u=P + 1), dict(token=Q + 2), dict(logprob=Q + 2), dict(temperature=P + 1),
               dict(top_k=P + 2), dict(top_p=P + 3), dict(min_p=P + 1)):
        _refused(1, call, **kw)
    _refused(2, call, shape=(2, rs.MAX_VOCAB + 1))
    _refused(2, call, shape=(1 << 31, 50))
    call(None, (0, 50), "bf16", None, None)
    call(None, (2, 0), "bf16", None, None)


def test_balance_refusals():
    assert rs.reshard_balance_loss_workspace((-1, 5, 6)) == 0
    need = rs.reshard_balance_loss_workspace((2, 5, 6))
    assert need > 0

    def call(logits=P, shape=(2, 5, 6), dtype="fp32", experts=P, topk=2, ws=P, counts=Q,
             workspace_bytes=need, **kw):
        rs.reshard_balance_loss(logits, shape, dtype, experts, topk, 0.1, ws, counts,
                                workspace_bytes=workspace_bytes, **kw)
    for kw in (dict(logits=None), dict(experts=None), dict(ws=None), dict(counts=None), dict(dtype="u8"),
               dict(score=7), dict(topk=0), dict(shape=(-2, 5, 6)), dict(shape=(2, -5, 6)),
               dict(shape=(2, 5, -6)), dict(ld=5), dict(workspace_bytes=need - 1), dict(ws=P + 4),
               dict(logits=P + 2), dict(dlogits=Q + 1), dict(experts=P + 1), dict(counts=Q + 2),
               dict(loss=Q + 1), dict(grad=P + 1)):
        _refused(1, call, **kw)
    _refused(2, call, shape=(2, 5, rs.MAX_EXPERTS + 1))
    _refused(2, call, shape=(1 << 20, 1 << 12, 6))


def test_oracle_e4m3():
    """The oracle's rounding against its table of values: every value is its own nearest,
    halves go to the even mantissa."""
    values = oo.e4m3_values()
    finite = np.unique(values[np.isfinite(values)])
    assert np.array_equal(oo.to_e4m3(finite), finite)
    assert len(finite) == 253 and finite[-1] == 448
    mid = (finite[1:] + finite[:-1]) / 2
    got = oo.to_e4m3(mid)
    assert np.all((got == finite[1:]) | (got == finite[:-1]))
    for v in got:
        b = int(np.flatnonzero(values == v)[0])
        assert b % 2 == 0, v
    assert np.array_equal(oo.to_e4m3(mid * (1 + 1e-9) + 0)[mid > 0], finite[1:][mid > 0])
    assert np.isnan(oo.to_e4m3(np.nan)) and oo.to_e4m3(1e9) == 448 and oo.to_e4m3(-1e9) == -448
