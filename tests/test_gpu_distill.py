"""Distillation from a teacher's most likely tokens on a GB300, loss and gradient, against plain
64-bit forms (logit_oracles), at the sizes, lists, alignments and masks where they can go wrong."""
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


def _check(x, dtype, token, y, tail, temperature=None, grad=None, ld=None, shift=0, other=0, inplace=False, rows=None):
    n, vocab = x.shape
    k = token.shape[1]
    ld = ld or vocab
    buf, view = _placed(x.cuda(), ld, shift, 50.0)
    if inplace:
        out, oview = buf, view
    else:
        out, oview = _placed(torch.full((n, vocab), 9.0, dtype=DT[dtype], device="cuda"), ld, other, 50.0)
    loss = torch.full((n,), 7.0, device="cuda")
    ltoken, ly = torch.full((n, k + 2), 3, dtype=torch.int32), torch.full((n, k + 2), 0.5)
    ltoken[:, :k], ly[:, :k] = token, y
    rs.reshard_distill_loss(buf, (n, vocab), dtype, ltoken.cuda(), ly.cuda(), k, loss=loss, dlogits=out, tail=tail,
                            temperature=None if temperature is None else temperature.cuda(),
                            grad=None if grad is None else grad.cuda(), ld=ld, ldtop=k + 2)
    torch.cuda.synchronize()
    assert bool((oview[:, vocab:] == 50.0).all())
    got = _f64(oview[:, :vocab])
    full = _f64(x)
    for r in range(n) if rows is None else rows:
        l, lb, g, gb = lo.distill(lo.cleaned(full[r], dtype), 1.0 if temperature is None else float(temperature[r]),
                                  token[r].numpy(), _f64(y[r]), tail, 1.0 if grad is None else float(grad[r]), EPS[dtype])
        assert float(loss[r]) == l or abs(float(loss[r]) - l) <= lb, (r, float(loss[r]), l, lb)
        worst = np.max(np.abs(got[r] - g) - gb)
        assert worst <= 0, (r, worst, int(np.argmax(np.abs(got[r] - g) - gb)))
    return loss, got


def _case(rows, vocab, k, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * 2
    n = min(20, vocab)
    x.scatter_add_(1, torch.randint(0, vocab, (rows, n), generator=g), 8 + 3 * torch.randn(rows, n, generator=g))
    temperature = torch.tensor([1.0, 0.7, 0.0, 1.9])[torch.randint(0, 4, (rows,), generator=g)]
    z = (x + torch.randn(rows, vocab, generator=g)) / torch.where(temperature > 0, temperature, 1.0)[:, None]
    top = torch.log_softmax(z, 1).topk(min(k, vocab), dim=1)
    token, y = top.indices.to(torch.int32), top.values
    if k > vocab:
        token = torch.nn.functional.pad(token, (0, k - vocab), value=-1)
        y = torch.nn.functional.pad(y, (0, k - vocab))
    return x, token, y, temperature, torch.rand(rows, generator=g) - 0.3


SHAPES = [(1, 1, 1), (2, 2, 3), (3, 7, 2), (5, 129, 129), (4, 1000, 50), (2, 16385, 64), (3, 50021, 1), (1, 131072, 256),
          (1, 262147, 33), (200, 333, 20), (170, 4099, 100), (31, 20000, 7)]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab,k", SHAPES)
def test_distill(rows, vocab, k, dtype, tail):
    x, token, y, temperature, grad = _case(rows, vocab, k, rows + vocab + k)
    if rows > 2:
        token[1] = -1                       # a row that does not count
        token[2, k // 2:] = vocab           # a short list
    if rows > 3:
        y[3, 0] = math.nan
    x = x.to(DT[dtype])
    pick = None if rows <= 5 else range(0, rows, rows // 6)
    _check(x, dtype, token, y, tail, temperature, grad, rows=pick)
    _check(x, dtype, token, y, tail, temperature, None, ld=vocab + 3, shift=1, other=1, rows=pick)
    _check(x, dtype, token, y, tail, None, grad, ld=vocab + 8, shift=0, other=1, rows=pick)
    _check(x, dtype, token, y, tail, temperature, grad, ld=vocab + 5, shift=3, inplace=True, rows=pick)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_largest_vocabulary(dtype, tail):
    x, token, y, temperature, grad = _case(1, rs.MAX_VOCAB, 64, 5)
    token[0, 0], token[0, 1] = 0, rs.MAX_VOCAB - 1
    _check(x.to(DT[dtype]), dtype, token, y, tail, temperature, grad)
    _check(x.to(DT[dtype]), dtype, token, y, tail, temperature, grad, inplace=True)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rows", [2, 300])
def test_tokens_that_stand_there_twice(rows, tail):
    vocab, k = 3001, 70
    x, token, y, temperature, grad = _case(rows, vocab, k, 8)
    token[:, 5], token[:, 6], token[:, 69] = token[:, 0], token[:, 1], token[:, 0]
    token[1, :] = 7
    y -= 1.0                                # sums below 1
    first = _check(x, "fp32", token, y, tail, temperature, grad, rows=range(0, rows, max(1, rows // 5)))
    for _ in range(3):
        again = _check(x, "fp32", token, y, tail, temperature, grad, rows=range(1))
        assert torch.equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_masks_nan_infinities_and_extremes(dtype, tail):
    big = lo.LARGEST[dtype]
    n, vocab, k = 11, 900, 6
    g = torch.Generator().manual_seed(4)
    x = torch.randn(n, vocab, generator=g)
    token = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(n)]).to(torch.int32)
    y = torch.log_softmax(torch.randn(n, k, generator=g), 1) - 0.2
    x[0, ::2] = -math.inf
    token[0] = torch.arange(k) * 2 + 1
    x[1, int(token[1, 0])] = -math.inf      # a likely token of the teacher's that the student has not
    x[2, :] = -math.inf
    x[3, 3] = math.nan
    x[4, 7] = math.inf
    x[5, 0], x[5, 1] = big, -big
    token[5, 0] = 0
    token[5, 1:] = -1
    y[6, :] = -math.inf
    y[7, 1:] = -math.inf
    x[8, :] = -math.inf
    x[8, token[8].long()] = 0.5             # nothing outside the list
    y[9] = -40.0
    token[10] = torch.tensor([0, vocab - 1, vocab, -5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    _check(x.to(DT[dtype]), dtype, token, y, tail)


def test_a_token_that_is_certain_gives_its_negative_log_likelihood():
    rows, vocab = 9, 2000
    x, token, _, temperature, _ = _case(rows, vocab, 1, 11)
    x, token, temperature = x.cuda(), token.cuda(), temperature.cuda()
    loss, dl = torch.empty(rows, device="cuda"), torch.empty(rows, vocab, device="cuda")
    rs.reshard_distill_loss(x, (rows, vocab), "fp32", token, torch.zeros(rows, 1, device="cuda"), 1, loss=loss,
                            dlogits=dl, temperature=temperature)
    lp, state, want = torch.empty(rows, device="cuda"), torch.empty(rows, 4, device="cuda"), torch.empty_like(dl)
    rs.reshard_logprob(x, (rows, vocab), "fp32", target=token, logprob=lp, state=state, temperature=temperature)
    rs.reshard_logprob_grad(x, (rows, vocab), "fp32", state, want, target=token,
                            dlogprob=torch.full((rows,), -1.0, device="cuda"), temperature=temperature)
    torch.cuda.synchronize()
    for r in range(rows):
        bound = lo.logprob(_f64(x[r]), float(temperature[r]), int(token[r]))[1]
        assert abs(float(loss[r]) + float(lp[r])) <= 3 * bound
        gb = lo.logprob_grad(_f64(x[r]), float(temperature[r]), int(token[r]), -1.0, 0.0, EPS["fp32"])[1]
        assert np.all(np.abs(_f64(dl[r]) - _f64(want[r])) <= 3 * gb)


def test_loss_or_gradient_alone():
    rows, vocab, k = 6, 5000, 20
    x, token, y, temperature, grad = _case(rows, vocab, k, 2)
    want, wgrad = _check(x, "fp32", token, y, True, temperature, grad)
    args = (x.cuda(), (rows, vocab), "fp32", token.cuda(), y.cuda(), k)
    kw = dict(tail=True, temperature=temperature.cuda(), grad=grad.cuda())
    loss, dl = torch.empty(rows, device="cuda"), torch.empty(rows, vocab, device="cuda")
    rs.reshard_distill_loss(*args, loss=loss, **kw)
    rs.reshard_distill_loss(*args, dlogits=dl, **kw)
    torch.cuda.synchronize()
    assert torch.equal(loss, want) and np.array_equal(_f64(dl), wgrad)


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(tail):
    """Central differences with steps of 2^-6: off by the step's square times a third derivative (at
    most 6 for a loss whose gradients are differences of probabilities) and by the losses' own bounds
    over the step."""
    rows, vocab, k, step = 3, 40, 5, 2.0 ** -6
    x, token, y, _, _ = _case(rows, vocab, k, 31)
    temperature = torch.tensor([1.0, 2.0, 1.5])
    y -= 0.1

    def value(a):
        loss = torch.empty(rows, device="cuda")
        rs.reshard_distill_loss(a.cuda(), (rows, vocab), "fp32", token.cuda(), y.cuda(), k, loss=loss, tail=tail,
                                temperature=temperature.cuda())
        return _f64(loss)
    _, grad = _check(x, "fp32", token, y, tail, temperature)
    for i in range(vocab):
        up, down = x.clone(), x.clone()
        up[:, i] += step
        down[:, i] -= step
        exact = _f64(up[:, i]) - _f64(down[:, i])
        slope = (value(up) - value(down)) / exact
        for r in range(rows):
            off = lo.distill(_f64(x[r]), float(temperature[r]), token[r].numpy(), _f64(y[r]), tail, 1.0, EPS["fp32"])[1]
            assert abs(slope[r] - grad[r, i]) <= 4 * off / exact[r] + 6 * step * step


def test_rows_far_apart():
    """Rows whose byte offsets pass 32 bits."""
    rows, vocab, ld, k = 3, 1000, 3 << 29, 8
    x, token, y, _, _ = _case(rows, vocab, k, 3)
    x = x.bfloat16()
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    view = buf.view(rows, ld)[:, :vocab]
    view.copy_(x)
    loss = torch.empty(rows, device="cuda")
    rs.reshard_distill_loss(buf, (rows, vocab), "bf16", token.cuda(), y.cuda(), k, loss=loss, dlogits=buf, ld=ld)
    torch.cuda.synchronize()
    for r in range(rows):
        l, lb, g, gb = lo.distill(_f64(x[r]), 1.0, token[r].numpy(), _f64(y[r]), False, 1.0, EPS["bf16"])
        assert abs(float(loss[r]) - l) <= lb and np.all(np.abs(_f64(view[r]) - g) <= gb)


def test_a_teachers_list_of_its_own_logits():
    """The alternatives that reshard_logprob lists serve as they are: a teacher that is the student has
    divergence 0 from itself, and with the rest as an outcome no gradient."""
    rows, vocab, k = 12, 6000, 30
    x, _, _, temperature, _ = _case(rows, vocab, k, 17)
    x, temperature = x.bfloat16().cuda(), temperature.cuda()
    token, y = torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, device="cuda")
    rs.reshard_logprob(x, (rows, vocab), "bf16", top_token=token, top_logprob=y, ntop=k, temperature=temperature)
    _, got = _check(x.cpu(), "bf16", token.cpu(), y.cpu(), True, temperature.cpu())
    assert np.max(np.abs(got)) < 1e-4
    _check(x.cpu(), "bf16", token.cpu(), y.cpu(), False, temperature.cpu())


def test_an_infinite_temperature_and_gradients_that_are_not_finite():
    rows, vocab, k = 4, 700, 9
    x, token, y, _, _ = _case(rows, vocab, k, 23)
    x[0, ::2] = -math.inf
    token[0] = torch.arange(k) * 2 + 1
    token[3] = -1
    temperature = torch.tensor([math.inf, math.inf, 1.0, 1.0])
    grad = torch.tensor([1.0, math.nan, math.inf, math.nan])
    loss, dl = torch.empty(rows, device="cuda"), torch.empty(rows, vocab, device="cuda")
    for tail in (False, True):
        rs.reshard_distill_loss(x.cuda(), (rows, vocab), "fp32", token.cuda(), y.cuda(), k, loss=loss, dlogits=dl,
                                tail=tail, temperature=temperature.cuda(), grad=grad.cuda())
        torch.cuda.synchronize()
        flat = x.clone()
        flat[0] = torch.where(flat[0] > -math.inf, 0.0, flat[0])
        want, bound, _, _ = lo.distill(_f64(flat[0]), 1.0, token[0].numpy(), _f64(y[0]), tail, 1.0, EPS["fp32"])
        assert abs(float(loss[0]) - want) <= bound
        assert bool(dl[0].isfinite().all()) and float(dl[0].abs().max()) <= 2.0 ** -120   # 1 / T
        assert bool(dl[1].isnan().all()) and not bool(dl[2].isfinite().any()) and bool((dl[3] == 0).all())


def test_a_value_that_is_infinite_is_not_taken_for_a_loss():
    x, token, y, _, _ = _case(2, 300, 5, 29)
    y[0, 1] = math.inf
    loss = torch.empty(2, device="cuda")
    rs.reshard_distill_loss(x.cuda(), (2, 300), "fp32", token.cuda(), y.cuda(), 5, loss=loss)
    torch.cuda.synchronize()
    assert math.isnan(float(loss[0])) and math.isfinite(float(loss[1]))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_rows_of_the_largest_vocabulary(dtype, tail):
    rows, vocab, k = 140, rs.MAX_VOCAB, 64
    g = torch.Generator(device="cuda").manual_seed(13)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(DT[dtype])
    y = torch.log_softmax(x.float() + torch.randn(rows, vocab, generator=g, device="cuda"), 1).topk(k, dim=1)
    token, value = y.indices.to(torch.int32), y.values.contiguous()
    loss, grad = torch.empty(rows, device="cuda"), torch.empty_like(x)
    rs.reshard_distill_loss(x, (rows, vocab), dtype, token, value, k, loss=loss, dlogits=grad, tail=tail)
    torch.cuda.synchronize()
    for r in (0, 70, 139):
        l, lb, want, bound = lo.distill(lo.cleaned(_f64(x[r]), dtype), 1.0, token[r].cpu().numpy(), _f64(value[r]), tail,
                                        1.0, EPS[dtype])
        assert abs(float(loss[r]) - l) <= lb
        assert np.all(np.abs(_f64(grad[r]) - want) <= bound)


@pytest.mark.parametrize("k", [1, 2, 64, 256])
@pytest.mark.parametrize("exponent", [10, 15, 20])
def test_a_small_rest(k, exponent):
    """What is left of 1 keeps its digits: its relative bound is 2^-21, 2^-41 of 1 at the smallest."""
    g = torch.Generator().manual_seed(k + exponent)
    n, vocab = 4, 5000
    x = torch.randn(n, vocab, generator=g)
    token = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(n)]).to(torch.int32)
    y = torch.log(torch.softmax(torch.randn(n, k, generator=g, dtype=torch.float64) * 2, 1)
                  * (1 - 2.0 ** -exponent)).float()
    x.scatter_(1, token.long(), y + 20.0)      # a student that knows most of it
    _check(x, "fp32", token, y, True)
    _check(x.bfloat16(), "bf16", token, y, True)
