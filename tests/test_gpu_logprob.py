"""Log-probabilities, entropies and alternatives of rows of logits on a GB300, and the gradient in
the logits, against plain 64-bit forms (logit_oracles), at the sizes, alignments, masks and orders
where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import logit_oracles as lo

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


def _placed(x, ld, shift, fill):
    r, c = x.shape
    buf = torch.full((shift + r * ld,), fill, dtype=x.dtype, device="cuda")
    view = buf[shift:].view(r, ld)
    view[:, :c] = x
    return buf[shift:], view


def _score(x, dtype, target, temperature, ntop, ld=None, shift=0, fill=50.0):
    """Calls with everything asked for; (logprob, entropy, tokens, their logprobs, state)."""
    rows, vocab = x.shape
    ld = ld or vocab
    buf, _ = _placed(x.cuda(), ld, shift, fill)
    logprob, entropy = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    token = torch.full((rows, ntop + 1), 77, dtype=torch.int32, device="cuda")
    top = torch.full((rows, ntop + 1), 77.0, device="cuda")
    state = torch.full((rows, 4), 7.0, device="cuda")
    rs.reshard_logprob(buf, (rows, vocab), dtype, target=target.cuda(), logprob=logprob, entropy=entropy,
                       top_token=token, top_logprob=top, ntop=ntop, state=state,
                       temperature=None if temperature is None else temperature.cuda(), ld=ld, ldtop=ntop + 1)
    torch.cuda.synchronize()
    assert bool((token[:, ntop] == 77).all()) and bool((top[:, ntop] == 77.0).all())
    return logprob, entropy, token[:, :ntop], top[:, :ntop], state


def _check_scores(x, dtype, target, temperature, ntop, **kw):
    logprob, entropy, token, top, state = _score(x, dtype, target, temperature, ntop, **kw)
    full = _f64(x)
    token, top = token.cpu().numpy(), _f64(top)
    for r in range(len(x)):
        y, t = lo.cleaned(full[r], dtype), 1.0 if temperature is None else float(temperature[r])
        at = int(target[r])
        if not 0 <= at < len(y):
            assert float(logprob[r]) == 0 and float(entropy[r]) == 0
            assert np.all(token[r] == -1) and np.all(top[r] == -np.inf)
            continue
        for got, (want, bound) in ((float(logprob[r]), lo.logprob(y, t, at)), (float(entropy[r]), lo.entropy(y, t))):
            assert got == want or abs(got - want) <= bound, (r, got, want, bound)
        want = lo.most_likely(y, ntop)
        assert np.array_equal(token[r], want), (r, token[r], want)
        for i in range(ntop):
            v, bound = lo.logprob(y, t, want[i]) if want[i] >= 0 else (-np.inf, 0.0)
            assert top[r, i] == v or abs(top[r, i] - v) <= bound, (r, i, top[r, i], v, bound)
    return state


def _logits(rows, vocab, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * 2
    n = min(20, vocab)
    x.scatter_add_(1, torch.randint(0, vocab, (rows, n), generator=g), 8 + 3 * torch.randn(rows, n, generator=g))
    target = torch.randint(0, vocab, (rows,), generator=g).to(torch.int32)
    temperature = torch.tensor([1.0, 0.7, 0.0, 1.9])[torch.randint(0, 4, (rows,), generator=g)]
    return x, target, temperature, g


SHAPES = [(1, 1), (2, 2), (3, 7), (5, 129), (4, 1000), (2, 16385), (3, 50021), (1, 131072), (1, 262147), (200, 333),
          (160, 4099), (33, 20000)]


@pytest.mark.parametrize("ntop", [0, 1, 20, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_scores(rows, vocab, dtype, ntop):
    x, target, temperature, g = _logits(rows, vocab, rows + vocab + ntop)
    if rows > 1:
        target[1] = -1
        target[-1] = vocab
    x = x.to(DT[dtype])
    for ld, shift in ((vocab, 0), (vocab + 3, 1)):
        _check_scores(x, dtype, target, temperature, ntop, ld=ld, shift=shift)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_the_largest_vocabulary(dtype):
    x, target, temperature, _ = _logits(1, rs.MAX_VOCAB, 3)
    _check_scores(x.to(DT[dtype]), dtype, target, temperature, 40)


def _orders(vocab, g):
    """Rows whose order, ties or masks are hard on a selection."""
    ramp = torch.arange(vocab) / vocab * 30
    few = torch.randint(0, 3, (vocab,), generator=g).float()
    rows = [ramp, -ramp, torch.zeros(vocab), torch.full((vocab,), -3.0), few, torch.randn(vocab, generator=g)]
    sparse = torch.full((vocab,), -math.inf)
    sparse[torch.randint(0, vocab, (9,), generator=g)] = torch.randn(9, generator=g)
    one = torch.full((vocab,), -math.inf)
    one[vocab - 1] = -7.0
    last = torch.cat([torch.full((vocab - vocab // 8,), -1e4), torch.randn(vocab // 8, generator=g)])
    zeros = torch.where(torch.rand(vocab, generator=g) < 0.5, 0.0, -0.0)
    stairs = (torch.arange(vocab) // 512 % 2).float() + torch.rand(vocab, generator=g) * 1e-3
    return torch.stack(rows + [sparse, one, torch.full((vocab,), -math.inf), last, zeros, stairs])


@pytest.mark.parametrize("copies", [1, 20])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [300, 9000, 50021])
def test_orders_ties_and_masks(vocab, dtype, copies):
    """copies: rows enough for one CTA a row, and few enough for several."""
    if copies > 1 and vocab > 9000:
        vocab = 20011
    g = torch.Generator().manual_seed(vocab)
    x = _orders(vocab, g)
    target = torch.randint(0, vocab, (len(x),), generator=g).to(torch.int32)
    target[7] = vocab - 1
    for ntop in (1, 100, 256):
        logprob, entropy, token, top, _ = _score(x.repeat(copies, 1).to(DT[dtype]), dtype, target.repeat(copies), None,
                                                 ntop)
        n = len(x)
        for c in range(copies):
            s = slice(c * n, (c + 1) * n)
            assert torch.equal(token[s], token[:n])
            # a row's sums are split at its granules of 16 aligned bytes: two rows that lie alike on
            # them are added up in the same order and give the same bits, others need not
            if c * n * vocab * DT[dtype].itemsize % 16 == 0:
                assert torch.equal(logprob[s], logprob[:n]) and torch.equal(entropy[s], entropy[:n])
                assert torch.equal(top[s], top[:n])
        _check_scores(x.to(DT[dtype]), dtype, target, None, ntop)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_nan_infinities_and_extremes(dtype):
    big = lo.LARGEST[dtype]
    x = torch.zeros(9, 700)
    x[0, 5] = math.nan
    x[1, 5] = math.inf
    x[2, [5, 600]] = math.inf
    x[3, :] = math.nan
    x[4, 0], x[4, 1] = big, -big
    x[5, :] = -big
    x[6, 10] = math.inf
    x[6, 11] = math.nan
    x[6, 12] = -math.inf
    x[7, :] = big
    x[8, :350] = -math.inf
    x[8, 350:] = math.nan
    x = x.to(DT[dtype])
    target = torch.tensor([5, 5, 600, 0, 1, 3, 12, 9, 400], dtype=torch.int32)
    for t in (None, torch.tensor([1.0, 1e-30, 1e30, -1.0, math.nan, 0.0, 3.0, 1e-42, 1.0])):
        _check_scores(x, dtype, target, t, 4)


def test_small_and_large_temperatures():
    x, target, _, _ = _logits(8, 3000, 9)
    t = torch.tensor([1e-40, 1e-10, 1e-3, 0.05, 20.0, 1e4, 1e20, 3e38])
    _check_scores(x, "fp32", target, t, 10)


def test_each_output_alone():
    rows, vocab = 5, 1003
    x, target, temperature, _ = _logits(rows, vocab, 4)
    want = dict(zip(("logprob", "entropy", "token", "top", "state"), _score(x, "fp32", target, temperature, 7)))
    x, target, temperature = x.cuda(), target.cuda(), temperature.cuda()
    for name in ("logprob", "entropy", "state", "top"):
        kw = {}
        if name == "top":
            kw = dict(top_token=torch.empty(rows, 7, dtype=torch.int32, device="cuda"),
                      top_logprob=torch.empty(rows, 7, device="cuda"), ntop=7)
        else:
            kw = {name: torch.empty_like(want[name])}
        rs.reshard_logprob(x, (rows, vocab), "fp32", target=target, temperature=temperature, **kw)
        torch.cuda.synchronize()
        if name == "top":
            assert torch.equal(kw["top_token"], want["token"]) and torch.equal(kw["top_logprob"], want["top"])
        else:
            assert torch.equal(kw[name], want[name])
    # without targets every row counts
    entropy = torch.empty(rows, device="cuda")
    rs.reshard_logprob(x, (rows, vocab), "fp32", entropy=entropy, temperature=temperature)
    torch.cuda.synchronize()
    assert torch.equal(entropy, want["entropy"])


def test_a_drawn_token_has_the_same_logprob():
    rows, vocab = 64, 5000
    x, _, temperature, _ = _logits(rows, vocab, 6)
    x, temperature = x.bfloat16().cuda(), temperature.cuda()
    token, drawn = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    rs.reshard_sample(x, (rows, vocab), "bf16", torch.rand(rows, device="cuda"), token, drawn, temperature=temperature)
    scored = torch.empty(rows, device="cuda")
    rs.reshard_logprob(x, (rows, vocab), "bf16", target=token, logprob=scored, temperature=temperature)
    torch.cuda.synchronize()
    for r in range(rows):
        y = lo.cleaned(_f64(x[r]), "bf16")
        want, bound = lo.logprob(y, float(temperature[r]), int(token[r]))
        assert abs(float(scored[r]) - want) <= bound and abs(float(drawn[r]) - want) <= 2 * bound


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_gradient(rows, vocab, dtype):
    x, target, temperature, g = _logits(rows, vocab, rows * 3 + vocab)
    if rows > 1:
        target[1] = -1
    x = x.to(DT[dtype])
    dl, dh = torch.randn(rows, generator=g), torch.randn(rows, generator=g) * 0.1
    if rows > 2:
        dl[2] = dh[2] = 0.0
    pick = range(rows) if rows <= 5 else range(0, rows, rows // 5)
    for ld, shift, other, inplace in ((vocab, 0, 0, False), (vocab + 3, 1, 1, False), (vocab + 8, 0, 1, False),
                                      (vocab + 5, 3, 0, True)):
        buf, view = _placed(x.cuda(), ld, shift, 50.0)
        state = torch.empty(rows, 4, device="cuda")
        kw = dict(target=target.cuda(), temperature=temperature.cuda(), ld=ld)
        rs.reshard_logprob(buf, (rows, vocab), dtype, state=state, **kw)
        for a, b in ((dl, dh), (dl, None), (None, dh)):
            if inplace:
                if b is None or a is None:
                    continue
                grad, gview = buf, view
            else:
                grad, gview = _placed(torch.full((rows, vocab), 9.0, dtype=DT[dtype], device="cuda"), ld, other, 50.0)
            rs.reshard_logprob_grad(buf, (rows, vocab), dtype, state, grad, dlogprob=None if a is None else a.cuda(),
                                    dentropy=None if b is None else b.cuda(), **kw)
            torch.cuda.synchronize()
            assert bool((gview[:, vocab:] == 50.0).all())
            got = _f64(gview[:, :vocab])
            for r in pick:
                ga, gb = 0.0 if a is None else float(a[r]), 0.0 if b is None else float(b[r])
                if int(target[r]) < 0 or (ga == 0 and gb == 0):
                    assert np.all(got[r] == 0)
                    continue
                want, bound = lo.logprob_grad(lo.cleaned(_f64(x[r]), dtype), float(temperature[r]), int(target[r]),
                                              ga, gb, EPS[dtype])
                assert np.all(np.abs(got[r] - want) <= bound), (r, np.max(np.abs(got[r] - want) / bound))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_gradient_of_masks_nan_and_infinities(dtype):
    big = lo.LARGEST[dtype]
    x = torch.randn(7, 900, generator=torch.Generator().manual_seed(2))
    x[0, ::2] = -math.inf
    x[1, :] = -math.inf
    x[2, 3] = math.nan
    x[3, 7] = math.inf
    x[4, 0], x[4, 1] = big, -big
    x[5, :] = math.nan
    x[6, 5] = -math.inf
    x = x.to(DT[dtype])
    target = torch.tensor([1, 0, 4, 8, 1, 2, 5], dtype=torch.int32)
    dl, dh = torch.full((7,), 1.5), torch.full((7,), -0.5)
    state, grad = torch.empty(7, 4, device="cuda"), torch.empty(7, 900, dtype=DT[dtype], device="cuda")
    rs.reshard_logprob(x.cuda(), (7, 900), dtype, target=target.cuda(), state=state)
    rs.reshard_logprob_grad(x.cuda(), (7, 900), dtype, state, grad, target=target.cuda(), dlogprob=dl.cuda(),
                            dentropy=dh.cuda())
    torch.cuda.synchronize()
    got = _f64(grad)
    for r in range(7):
        want, bound = lo.logprob_grad(lo.cleaned(_f64(x[r]), dtype), 1.0, int(target[r]), 1.5, -0.5, EPS[dtype])
        assert np.all(np.abs(got[r] - want) <= bound), r


def test_gradient_against_differences():
    """Central differences of the float64 sum of outputs with steps of 2^-6: off by the step's square
    times a third derivative (each at most 6 times the gradients' sizes here) and by the outputs'
    own bounds over the step."""
    rows, vocab, step = 3, 40, 2.0 ** -6
    x, target, _, g = _logits(rows, vocab, 12)
    temperature = torch.tensor([1.0, 2.0, 1.5])
    dl, dh = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    target, tcuda = target.cuda(), temperature.cuda()

    def value(y):
        lp, h = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        rs.reshard_logprob(y.cuda(), (rows, vocab), "fp32", target=target, logprob=lp, entropy=h, temperature=tcuda)
        return _f64(lp) * _f64(dl) + _f64(h) * _f64(dh)
    state, grad = torch.empty(rows, 4, device="cuda"), torch.empty(rows, vocab, device="cuda")
    rs.reshard_logprob(x.cuda(), (rows, vocab), "fp32", target=target, state=state, temperature=tcuda)
    rs.reshard_logprob_grad(x.cuda(), (rows, vocab), "fp32", state, grad, target=target, dlogprob=dl.cuda(),
                            dentropy=dh.cuda(), temperature=tcuda)
    torch.cuda.synchronize()
    grad = _f64(grad)
    for i in range(vocab):
        up, down = x.clone(), x.clone()
        up[:, i] += step
        down[:, i] -= step
        exact = _f64(up[:, i]) - _f64(down[:, i])
        slope = (value(up) - value(down)) / exact
        for r in range(rows):
            y = _f64(x[r])
            t = float(temperature[r])
            off = 2 * (abs(float(dl[r])) * lo.logprob(y, t, int(target[r]))[1] + abs(float(dh[r])) * lo.entropy(y, t)[1])
            size = abs(float(dl[r])) + abs(float(dh[r])) * (4 + math.log(vocab))
            assert abs(slope[r] - grad[r, i]) <= 2 * off / exact[r] + 6 * size * step * step


def test_rows_far_apart():
    """Rows whose byte offsets pass 32 bits."""
    rows, vocab, ld = 3, 1000, 3 << 29
    x, target, _, _ = _logits(rows, vocab, 8)
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    view = buf.view(rows, ld)[:, :vocab]
    view.copy_(x.bfloat16())
    lp, state, token = (torch.empty(rows, device="cuda"), torch.empty(rows, 4, device="cuda"),
                        torch.empty(rows, 3, dtype=torch.int32, device="cuda"))
    kw = dict(target=target.cuda(), ld=ld)
    rs.reshard_logprob(buf, (rows, vocab), "bf16", logprob=lp, state=state, top_token=token,
                       top_logprob=torch.empty(rows, 3, device="cuda"), ntop=3, **kw)
    rs.reshard_logprob_grad(buf, (rows, vocab), "bf16", state, buf, dlogprob=torch.ones(rows, device="cuda"), **kw)
    torch.cuda.synchronize()
    for r in range(rows):
        y = lo.cleaned(_f64(x[r].bfloat16()), "bf16")
        want, bound = lo.logprob(y, 1.0, int(target[r]))
        assert abs(float(lp[r]) - want) <= bound
        assert np.array_equal(token[r].cpu().numpy(), lo.most_likely(y, 3))
        want, bound = lo.logprob_grad(y, 1.0, int(target[r]), 1.0, 0.0, EPS["bf16"])
        assert np.all(np.abs(_f64(view[r]) - want) <= bound)


def test_an_infinite_temperature_and_no_vocabulary():
    x = torch.randn(3, 500, generator=torch.Generator().manual_seed(3))
    x[1, ::3] = -math.inf
    x[2, 7] = math.nan
    target = torch.tensor([4, 1, 9], dtype=torch.int32)
    logprob, entropy, _, _, _ = _score(x, "fp32", target, torch.full((3,), math.inf), 0)
    counts = [500, 500 - 167, 499]        # all that count are as likely as each other
    for r in range(3):
        want = math.log(counts[r])
        # ln S of S equal ones, S exact: two roundings of the logarithm, and one of the result
        assert abs(float(logprob[r]) + want) <= 4 * 2.0 ** -24 * want
        assert abs(float(entropy[r]) - want) <= 4 * 2.0 ** -24 * want
    lp, token = torch.full((2,), 5.0, device="cuda"), torch.full((2, 3), 5, dtype=torch.int32, device="cuda")
    top = torch.full((2, 3), 5.0, device="cuda")
    rs.reshard_logprob(None, (2, 0), "bf16", target=torch.zeros(2, dtype=torch.int32, device="cuda"), logprob=lp,
                       top_token=token, top_logprob=top, ntop=3)
    torch.cuda.synchronize()
    assert bool((lp == 0).all()) and bool((token == -1).all()) and bool((top == -math.inf).all())


def test_gradients_that_are_not_finite_stay_so():
    x = torch.randn(5, 300, generator=torch.Generator().manual_seed(5))
    x[4] = -math.inf
    target = torch.tensor([1, 2, 3, -1, 5], dtype=torch.int32)
    dl = torch.tensor([math.nan, math.inf, 1.0, math.nan, math.nan])
    state, grad = torch.empty(5, 4, device="cuda"), torch.empty(5, 300, device="cuda")
    rs.reshard_logprob(x.cuda(), (5, 300), "fp32", target=target.cuda(), state=state)
    rs.reshard_logprob_grad(x.cuda(), (5, 300), "fp32", state, grad, target=target.cuda(), dlogprob=dl.cuda())
    torch.cuda.synchronize()
    assert bool(grad[0].isnan().all())
    assert not bool(grad[1].isfinite().any())
    assert bool(grad[2].isfinite().all())
    assert bool((grad[3:] == 0).all())       # rows that do not count, or have no finite logit


@pytest.mark.parametrize("dtype,ntop", [("fp32", 20), ("bf16", 100), ("fp16", 256)])
def test_many_rows_of_the_largest_vocabulary(dtype, ntop):
    """One CTA a row, whose threads note groups of several rounds."""
    rows, vocab = 140, rs.MAX_VOCAB
    g = torch.Generator(device="cuda").manual_seed(12)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(DT[dtype])
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    lp, h = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    token, top = (torch.empty(rows, ntop, dtype=torch.int32, device="cuda"), torch.empty(rows, ntop, device="cuda"))
    state, grad = torch.empty(rows, 4, device="cuda"), torch.empty_like(x)
    rs.reshard_logprob(x, (rows, vocab), dtype, target=target, logprob=lp, entropy=h, top_token=token,
                       top_logprob=top, ntop=ntop, state=state)
    rs.reshard_logprob_grad(x, (rows, vocab), dtype, state, grad, target=target,
                            dlogprob=torch.ones(rows, device="cuda"))
    torch.cuda.synchronize()
    for r in (0, 77, 139):
        y = lo.cleaned(_f64(x[r]), dtype)
        for got, (want, bound) in ((lp[r], lo.logprob(y, 1.0, int(target[r]))), (h[r], lo.entropy(y, 1.0))):
            assert abs(float(got) - want) <= bound
        best = lo.most_likely(y, ntop)
        assert np.array_equal(token[r].cpu().numpy(), best)
        bound = max(lo.logprob(y, 1.0, int(t))[1] for t in best[::10])
        z, _, normal, _, _ = lo.softmax(y, 1.0)
        assert np.all(np.abs(_f64(top[r]) - (z[best] - normal)) <= 2 * bound)
        want, bound = lo.logprob_grad(y, 1.0, int(target[r]), 1.0, 0.0, EPS[dtype])
        assert np.all(np.abs(_f64(grad[r]) - want) <= bound)
