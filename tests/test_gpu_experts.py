"""Sorting by expert, dispatch and combination of rows on a GB300, against plain 64-bit forms
(expert_oracles), at the sizes, pitches, alignments and choices where they can go wrong."""
import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import expert_oracles as eo

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half a unit in the last place of a result (finfo.eps / 2), and of the smallest one
EPS = {"bf16": (2.0 ** -8, 0.0), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (2.0 ** -24, 0.0)}


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    yield
    assert rs.reshard_device_status(clear=True) == 0


def _f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _sorted(experts, nexperts):
    t, k = experts.shape
    slot = torch.full((t, k), 77, dtype=torch.int32, device="cuda")
    offsets = torch.full((nexperts + 2,), 77, dtype=torch.int32, device="cuda")
    rs.reshard_expert_sort(experts.cuda(), (t, k), nexperts, slot, offsets)
    torch.cuda.synchronize()
    assert int(offsets[-1]) == 77
    return slot.cpu().numpy(), offsets[:-1].cpu().numpy()


@pytest.mark.parametrize("tokens,topk,nexperts", [
    (1, 1, 1), (1, 8, 256), (33, 2, 3), (31, 5, 7), (100, 8, 64), (1000, 3, 1), (1365, 6, 300),
    (1024, 8, 256), (1025, 8, 256), (5000, 2, 4096), (20000, 8, 1600), (9000, 1, 3000)])
@pytest.mark.parametrize("kind", ["uniform", "one", "rising", "dropped"])
def test_sort(tokens, topk, nexperts, kind):
    g = torch.Generator().manual_seed(tokens + topk + nexperts)
    e = torch.randint(0, nexperts, (tokens, topk), generator=g, dtype=torch.int32)
    if kind == "one":
        e[:] = nexperts - 1
    elif kind == "rising":
        e = (torch.arange(tokens * topk) * nexperts // (tokens * topk)).to(torch.int32).view(tokens, topk)
    elif kind == "dropped":
        e[torch.rand(e.shape, generator=g) < 0.3] = -1
        e[torch.rand(e.shape, generator=g) < 0.1] = nexperts
        e[torch.rand(e.shape, generator=g) < 0.1] = -2 ** 31
    slot, offsets = _sorted(e, nexperts)
    flat = e.numpy().reshape(-1)
    valid = (flat >= 0) & (flat < nexperts)
    order = np.argsort(np.where(valid, flat, nexperts), kind="stable")
    want = np.full(flat.shape, -1, np.int64)
    want[order[:valid.sum()]] = np.arange(valid.sum())
    assert np.array_equal(slot.reshape(-1), want)
    counts = np.bincount(flat[valid], minlength=nexperts)
    assert np.array_equal(offsets, np.concatenate([[0], np.cumsum(counts)]))


def test_sort_small_against_the_definition():
    g = torch.Generator().manual_seed(3)
    e = torch.randint(-1, 6, (17, 3), generator=g, dtype=torch.int32)
    slot, offsets = _sorted(e, 5)
    want = eo.sort(e.numpy(), 5)
    assert np.array_equal(slot, want[0]) and np.array_equal(offsets, want[1])


def test_sort_without_choices_or_experts():
    offsets = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    rs.reshard_expert_sort(None, (0, 3), 5, None, offsets)
    assert offsets.tolist() == [0] * 6
    offsets.fill_(9)
    rs.reshard_expert_sort(None, (3, 0), 4, None, offsets)
    assert offsets.tolist() == [0] * 5 + [9]
    slot = torch.full((4, 2), 5, dtype=torch.int32, device="cuda")
    rs.reshard_expert_sort(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), (4, 2), 0, slot, offsets)
    assert bool((slot == -1).all()) and int(offsets[0]) == 0


def _placed(x, ld, shift, fill):
    """x [r, c] in rows of ld elements, `shift` elements past an aligned address."""
    r, c = x.shape
    buf = torch.full((shift + r * ld,), fill, dtype=x.dtype, device="cuda")
    view = buf[shift:].view(r, ld)
    view[:, :c] = x
    return buf[shift:], view


def _slots(tokens, topk, nrows, g, dropped=0.2):
    """Different slots for all choices, some of them outside the rows."""
    n = tokens * topk
    slot = torch.randperm(max(n, nrows), generator=g)[:n].to(torch.int32)
    slot[slot >= nrows] = -1
    slot[torch.rand(n, generator=g) < dropped] = -1
    far = torch.rand(n, generator=g) < 0.05
    slot[far] = torch.tensor([nrows, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 3, (int(far.sum()),), generator=g)].to(torch.int32)
    return slot.view(tokens, topk)


SHAPES = [(1, 1, 1, 1), (1, 8, 7168, 8), (3, 2, 8, 7), (5, 3, 129, 15), (37, 8, 1000, 300), (9, 11, 4098, 120),
          (130, 1, 24, 130), (7, 2, 9001, 20), (600, 4, 72, 2400)]
LAYOUTS = [(0, 0, 0), (8, 8, 8), (1, 3, 1), (4, 2, 2)]   # extra pitch of x and of rows, shift


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,topk,cols,nrows", SHAPES)
def test_dispatch_combine_and_gradients(tokens, topk, cols, nrows, dtype, layout):
    g = torch.Generator().manual_seed(tokens * 7 + cols)
    px, pr, shift = layout
    slot = _slots(tokens, topk, nrows, g)
    x = torch.randn(tokens, cols, generator=g).to(DT[dtype]).cuda()
    shape, dslot = (tokens, topk, cols), slot.cuda()
    kw = dict(nrows=nrows, ldr=cols + pr)
    # dispatch
    xin, _ = _placed(x, cols + px, shift, 9.0)
    rows, view = _placed(torch.full((nrows, cols), 5.0, dtype=DT[dtype], device="cuda"), cols + pr, shift, 7.0)
    rs.reshard_expert_dispatch(xin, shape, dtype, dslot, rows, ldx=cols + px, **kw)
    torch.cuda.synchronize()
    want = torch.full((nrows, cols), 5.0, dtype=DT[dtype], device="cuda")
    for t in range(tokens):
        for j in range(topk):
            if 0 <= slot[t, j] < nrows:
                want[slot[t, j]] = x[t]
    assert torch.equal(view[:, :cols], want) and bool((view[:, cols:] == 7.0).all())
    # combine
    r = torch.randn(nrows, cols, generator=g).to(DT[dtype]).cuda()
    rin, _ = _placed(r, cols + pr, shift, 9.0)
    for weight in (None, torch.randn(tokens, topk, generator=g)):
        w = None if weight is None else weight.cuda()
        out, oview = _placed(torch.full((tokens, cols), 5.0, dtype=DT[dtype], device="cuda"), cols + px, shift, 7.0)
        rs.reshard_expert_combine(rin, shape, dtype, dslot, out, weight=w, ldo=cols + px, **kw)
        torch.cuda.synchronize()
        o, bound = eo.combine(_f64(r), slot.numpy(), None if weight is None else _f64(weight), EPS[dtype])
        assert np.all(np.abs(_f64(oview[:, :cols]) - o) <= bound)
        assert bool((oview[:, cols:] == 7.0).all())
        # gradients: both, and each alone
        d = torch.randn(tokens, cols, generator=g).to(DT[dtype]).cuda()
        din, _ = _placed(d, cols + px, shift, 9.0)
        wr, br, ww, bw = eo.combine_grad(_f64(d), _f64(r), slot.numpy(), None if weight is None else _f64(weight),
                                         EPS[dtype])
        for which in (3, 1, 2):
            drows, dview = _placed(torch.full((nrows, cols), 5.0, dtype=DT[dtype], device="cuda"), cols + pr,
                                   shift, 7.0)
            dweight = torch.full((tokens, topk), 5.0, device="cuda")
            rs.reshard_expert_combine_grad(din, shape, dtype, dslot, rows=rin if which & 2 else None, weight=w,
                                           drows=drows if which & 1 else None,
                                           dweight=dweight if which & 2 else None, ldo=cols + px, **kw)
            torch.cuda.synchronize()
            got = _f64(dview[:, :cols])
            left = np.isnan(wr)
            if which & 1:
                assert np.all(got[left] == 5.0) and np.all(np.abs(got - wr)[~left] <= br[~left])
            else:
                assert np.all(got == 5.0)
            assert bool((dview[:, cols:] == 7.0).all())
            if which & 2:
                assert np.all(np.abs(_f64(dweight) - ww) <= bw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,topk,cols,nrows", SHAPES)
def test_dispatch_in_8_bits_is_the_quantisation_of_each_row(tokens, topk, cols, nrows, dtype):
    g = torch.Generator().manual_seed(tokens * 5 + cols)
    slot = _slots(tokens, topk, nrows, g)
    x = (torch.randn(tokens, cols, generator=g) * 3).to(DT[dtype]).cuda()
    x[0, 0] = float("nan")
    x[-1, -1] = float("inf")
    B = -(-cols // 128)
    q = torch.empty(tokens, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(tokens, B, device="cuda")
    rs.reshard_fp8_quantize(x, q, s, (tokens, cols), dtype)
    for px, pr, shift in ((0, 0, 0), (8, 16, 8), (1, 3, 1)):
        xin, _ = _placed(x, cols + px, shift, 9.0)
        rows, view = _placed(torch.full((nrows, cols), 0xA5, dtype=torch.uint8, device="cuda"), cols + pr, shift, 0x5A)
        scale = torch.full((nrows, B + px), -5.0, device="cuda")
        rs.reshard_expert_dispatch(xin, (tokens, topk, cols), dtype, slot.cuda(), rows, scale=scale, nrows=nrows,
                                   ldx=cols + px, ldr=cols + pr, lds=B + px)
        torch.cuda.synchronize()
        wq = torch.full((nrows, cols), 0xA5, dtype=torch.uint8, device="cuda")
        ws = torch.full((nrows, B), -5.0, device="cuda")
        for t in range(tokens):
            for j in range(topk):
                if 0 <= slot[t, j] < nrows:
                    wq[slot[t, j]], ws[slot[t, j]] = q[t], s[t]
        assert torch.equal(view[:, :cols], wq) and bool((view[:, cols:] == 0x5A).all())
        assert torch.equal(scale[:, :B].view(torch.int32), ws.view(torch.int32))
        assert bool((scale[:, B:] == -5.0).all())


def test_rows_far_apart():
    """Places whose byte offsets pass 32 bits."""
    cols, ld = 64, 1 << 22
    nrows = 700
    rows = torch.zeros(nrows * ld, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(2, cols, device="cuda").bfloat16()
    slot = torch.tensor([[0, nrows - 1], [5, 650]], dtype=torch.int32, device="cuda")
    rs.reshard_expert_dispatch(x, (2, 2, cols), "bf16", slot, rows, nrows=nrows, ldr=ld)
    v = rows.view(nrows, ld)[:, :cols]
    for t in range(2):
        for j in range(2):
            assert torch.equal(v[slot[t, j]], x[t])
    out = torch.empty(2, cols, dtype=torch.bfloat16, device="cuda")
    rs.reshard_expert_combine(rows, (2, 2, cols), "bf16", slot, out, nrows=nrows, ldr=ld)
    assert torch.equal(out, (2 * x.float()).bfloat16())
    dw = torch.empty(2, 2, device="cuda")
    rs.reshard_expert_combine_grad(x, (2, 2, cols), "bf16", slot, rows=rows, dweight=dw, nrows=nrows, ldr=ld)
    want = (x.double() ** 2).sum(1)
    assert bool(((dw.double() - want[:, None]).abs() <= 26 * 2.0 ** -24 * want[:, None]).all())


def test_gradients_against_differences():
    """The combination is linear in rows and in weights: differences of any size give its slope."""
    t, k, c = 6, 3, 40
    g = torch.Generator().manual_seed(1)
    slot = torch.randperm(t * k, generator=g).to(torch.int32).view(t, k)
    slot[2, 1] = -1
    rows, w = torch.randn(t * k, c, generator=g).cuda(), torch.randn(t, k, generator=g).cuda()
    dout, dslot = torch.randn(t, c, generator=g).cuda(), slot.cuda()

    def value(r, weight):
        out = torch.empty(t, c, device="cuda")
        rs.reshard_expert_combine(r, (t, k, c), "fp32", dslot, out, weight=weight)
        return float((out.double() * dout.double()).sum())
    drows, dweight = torch.zeros(t * k, c, device="cuda"), torch.empty(t, k, device="cuda")
    rs.reshard_expert_combine_grad(dout, (t, k, c), "fp32", dslot, rows=rows, weight=w, drows=drows, dweight=dweight)
    torch.cuda.synchronize()
    # values are sums of t * c products of three numbers below 5, each rounded to 2^-24 of itself
    most = 2.0 ** -24 * (k + 2) * t * c * 125
    for i, j in ((0, 0), (2, 1), (5, 2)):
        step = torch.zeros_like(w)
        step[i, j] = 1.0
        assert abs(value(rows, w + step) - value(rows, w - step) - 2 * float(dweight[i, j])) <= 4 * most
    for i, j in ((0, 0), (7, 39), (17, 5)):
        step = torch.zeros_like(rows)
        step[i, j] = 1.0
        assert abs(value(rows + step, w) - value(rows - step, w) - 2 * float(drows[i, j])) <= 4 * most


def test_dispatch_gradient_is_a_combination_without_weights():
    """<rows, drows> = <x, dx> for the linear map x -> rows."""
    t, k, c, e = 50, 4, 96, 12
    g = torch.Generator(device="cuda").manual_seed(2)
    experts = torch.rand(t, e, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    experts[3] = -1
    slot, offsets = torch.empty(t, k, dtype=torch.int32, device="cuda"), torch.empty(e + 1, dtype=torch.int32, device="cuda")
    rs.reshard_expert_sort(experts, (t, k), e, slot, offsets)
    x = torch.randn(t, c, generator=g, device="cuda")
    rows, drows = torch.zeros(t * k, c, device="cuda"), torch.randn(t * k, c, generator=g, device="cuda")
    rs.reshard_expert_dispatch(x, (t, k, c), "fp32", slot, rows)
    dx = torch.empty(t, c, device="cuda")
    rs.reshard_expert_combine(drows, (t, k, c), "fp32", slot, dx)
    a, b = (rows.double() * drows.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(float(a - b)) <= k * 2.0 ** -24 * float((rows.double() * drows.double()).abs().sum())
    assert bool((dx[3] == 0).all()) and int(offsets[-1]) == (t - 1) * k


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols,pad", [(7168, 0), (7176, 0), (7172, 1), (5100, 3), (9216, 0), (2049, 0)])
def test_many_tokens(cols, pad, dtype):
    """Tokens enough for the kernels that take several blocks of a row a lane, or a whole row a CTA."""
    tokens, topk = 2100, 3
    nrows = tokens * topk
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn(tokens, cols, generator=g, device="cuda") * 3).to(DT[dtype])
    slot = torch.randperm(nrows, generator=g, device="cuda").to(torch.int32).view(tokens, topk)
    slot[5, 1] = -1
    shape, kw = (tokens, topk, cols), dict(ldr=cols + pad)
    xin, _ = _placed(x, cols + pad, pad, 9.0)
    at = slot.long().flatten()
    ok = at >= 0
    token = torch.arange(tokens, device="cuda").repeat_interleave(topk)
    # as they are
    rows, view = _placed(torch.full((nrows, cols), 5.0, dtype=DT[dtype], device="cuda"), cols + pad, pad, 7.0)
    rs.reshard_expert_dispatch(xin, shape, dtype, slot, rows, ldx=cols + pad, **kw)
    want = torch.full((nrows, cols), 5.0, dtype=DT[dtype], device="cuda")
    want[at[ok]] = x[token[ok]]
    assert torch.equal(view[:, :cols], want) and bool((view[:, cols:] == 7.0).all())
    # in 8 bits
    B = -(-cols // 128)
    q, s = torch.empty(tokens, cols, dtype=torch.uint8, device="cuda"), torch.empty(tokens, B, device="cuda")
    rs.reshard_fp8_quantize(x, q, s, (tokens, cols), dtype)
    rows8, view8 = _placed(torch.full((nrows, cols), 0xA5, dtype=torch.uint8, device="cuda"), cols + pad, pad, 0x5A)
    scale = torch.full((nrows, B), -5.0, device="cuda")
    rs.reshard_expert_dispatch(xin, shape, dtype, slot, rows8, scale=scale, ldx=cols + pad, **kw)
    want8, wants = torch.full_like(view8[:, :cols], 0xA5), torch.full_like(scale, -5.0)
    want8[at[ok]], wants[at[ok]] = q[token[ok]], s[token[ok]]
    assert torch.equal(view8[:, :cols], want8) and bool((view8[:, cols:] == 0x5A).all()) and torch.equal(scale, wants)
    # and back, with gradients: the bounds of expert_oracles
    w = torch.randn(tokens, topk, generator=g, device="cuda")
    out, oview = _placed(torch.full((tokens, cols), 5.0, dtype=DT[dtype], device="cuda"), cols + pad, pad, 7.0)
    rs.reshard_expert_combine(rows, shape, dtype, slot, out, weight=w, ldo=cols + pad, **kw)
    terms = torch.where(ok.view(tokens, topk, 1), x.double()[:, None] * w.double()[..., None], 0.0)
    total, size = terms.sum(1), terms.abs().sum(1)
    err = topk * 2.0 ** -24 * size
    assert bool(((oview[:, :cols].double() - total).abs() <= err + EPS[dtype][0] * (total.abs() + err)
                 + EPS[dtype][1]).all())
    assert bool((oview[:, cols:] == 7.0).all())
    drows, dview = _placed(torch.full((nrows, cols), 5.0, dtype=DT[dtype], device="cuda"), cols + pad, pad, 7.0)
    dw = torch.empty(tokens, topk, device="cuda")
    rs.reshard_expert_combine_grad(xin, shape, dtype, slot, rows=rows, weight=w, drows=drows, dweight=dw,
                                   ldo=cols + pad, **kw)
    # (exact products of the type's values by w, rounded to float32 and to the type)
    grad = torch.full((nrows, cols), 5.0, dtype=torch.float64, device="cuda")
    grad[at[ok]] = (x.double()[token] * w.double().flatten()[:, None])[ok]
    assert bool(((dview[:, :cols].double() - grad).abs() <= (EPS[dtype][0] + 2.0 ** -23) * grad.abs()
                 + EPS[dtype][1]).all())
    dots = torch.where(ok.view(tokens, topk), (x.double() ** 2).sum(1)[:, None], 0.0)
    assert bool(((dw.double() - dots).abs() <= (cols / 32 + 24) * 2.0 ** -24 * dots).all())
    assert bool((dview[:, cols:] == 7.0).all())
