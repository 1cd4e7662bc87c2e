"""Argument checks of sorting by expert, dispatch and combination, without a GPU: every refusal
comes before any device work, with a message, and calls with nothing to do are accepted."""
import pytest

import dtensor_reshard_gb300 as rs

P, Q = 0x10000, 0x20000     # addresses that are never dereferenced
INVALID, UNSUPPORTED = 1, 2


def _refused(status, call, *args, **kw):
    with pytest.raises(rs.ReshardError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    assert rs.reshard_last_error()


def test_sort_refusals():
    def call(experts=P, shape=(4, 2), nexperts=8, slot=Q, offsets=Q):
        rs.reshard_expert_sort(experts, shape, nexperts, slot, offsets)
    for kw in (dict(experts=None), dict(slot=None), dict(offsets=None), dict(shape=(-1, 2)), dict(shape=(4, -2)),
               dict(nexperts=-1), dict(experts=P + 2), dict(slot=Q + 1), dict(offsets=Q + 2)):
        _refused(INVALID, call, **kw)
    for kw in (dict(nexperts=rs.MAX_EXPERTS + 1), dict(shape=(1 << 30, 2)), dict(shape=(1 << 62, 1 << 62)),
               dict(shape=(1, 1 << 31))):
        _refused(UNSUPPORTED, call, **kw)


SIZES = [(1 << 31, 1, 8), (1, 1 << 31, 8), (1, 1, 1 << 31), (1 << 16, 1 << 15, 8), (1 << 62, 1 << 62, 8)]


@pytest.mark.parametrize("scale", [None, P])
def test_dispatch_refusals(scale):
    def call(x=P, shape=(4, 2, 64), dtype="bf16", slot=P, rows=Q, scale=scale, **kw):
        rs.reshard_expert_dispatch(x, shape, dtype, slot, rows, scale=scale, **kw)
    for kw in (dict(x=None), dict(slot=None), dict(rows=None), dict(dtype="i32"), dict(shape=(-4, 2, 64)),
               dict(shape=(4, -2, 64)), dict(shape=(4, 2, -64)), dict(nrows=-1), dict(ldx=63), dict(ldr=63),
               dict(x=P + 1), dict(slot=P + 2)):
        _refused(INVALID, call, **kw)
    if scale:
        _refused(INVALID, call, lds=0)
        _refused(INVALID, call, scale=P + 2)
    else:
        _refused(INVALID, call, rows=Q + 1)
    for shape in SIZES:
        _refused(UNSUPPORTED, call, shape=shape, nrows=4)
    _refused(UNSUPPORTED, call, nrows=1 << 31)
    _refused(UNSUPPORTED, call, shape=((1 << 31) - 1, 1, (1 << 31) - 64), nrows=4)   # the grid
    for kw in (dict(shape=(0, 2, 64)), dict(shape=(4, 0, 64)), dict(shape=(4, 2, 0)), dict(nrows=0)):
        call(None, slot=None, rows=None, **kw)


def test_combine_refusals():
    def call(rows=P, shape=(4, 2, 64), dtype="bf16", slot=P, out=Q, **kw):
        rs.reshard_expert_combine(rows, shape, dtype, slot, out, **kw)
    for kw in (dict(rows=None), dict(slot=None), dict(out=None), dict(dtype="u8"), dict(shape=(-4, 2, 64)),
               dict(shape=(4, -2, 64)), dict(shape=(4, 2, -64)), dict(nrows=-1), dict(ldo=63), dict(ldr=63),
               dict(rows=P + 1), dict(slot=P + 2), dict(out=Q + 1), dict(weight=P + 1)):
        _refused(INVALID, call, **kw)
    for shape in SIZES:
        _refused(UNSUPPORTED, call, shape=shape, nrows=4)
    for kw in (dict(shape=(0, 2, 64)), dict(shape=(4, 2, 0))):
        call(None, slot=None, out=None, **kw)


def test_combine_grad_refusals():
    def call(dout=P, shape=(4, 2, 64), dtype="bf16", slot=P, rows=P, drows=Q, dweight=Q, **kw):
        rs.reshard_expert_combine_grad(dout, shape, dtype, slot, rows=rows, drows=drows, dweight=dweight, **kw)
    for kw in (dict(dout=None), dict(slot=None), dict(rows=None), dict(dtype="i64"), dict(shape=(-4, 2, 64)),
               dict(shape=(4, -2, 64)), dict(shape=(4, 2, -64)), dict(nrows=-1), dict(ldo=63), dict(ldr=63),
               dict(rows=P + 1), dict(slot=P + 2), dict(dout=P + 1), dict(drows=Q + 1), dict(dweight=Q + 2),
               dict(weight=P + 1)):
        _refused(INVALID, call, **kw)
    for shape in SIZES:
        _refused(UNSUPPORTED, call, shape=shape, nrows=4)
    call(None, slot=None, rows=None, drows=None, dweight=None)
    for kw in (dict(shape=(0, 2, 64)), dict(shape=(4, 0, 64))):
        call(None, slot=None, rows=None, **kw)
