"""Values and sizes at the ends of the operators' ranges, against the 64-bit forms."""
import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import operator_oracles as oo
from tests.test_gpu_operators import DT, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    yield
    assert rs.reshard_device_status(clear=True) == 0


# --------------------------------------------------------------------------- quantize
def _bytes(values, negative):
    """The e4m3 bytes of values with the given signs (of zeros too)."""
    table = oo.e4m3_values()[:127]
    return np.searchsorted(table, np.abs(values)).astype(np.uint8) | (negative.astype(np.uint8) << 7)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [256, 203])
def test_quantize_keeps_the_sign_of_zeros(cols, dtype, block_rows):
    """x / scale is -0 where x is, and rounds to -0 where x is small and negative."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(150, cols, generator=g, device="cuda")
    x[:, ::3] = -0.0
    x[:, 1::9] = 0.0
    x[:, 2::9] *= 1e-4
    x[5] = -0.0                              # (blocks of zeros alone)
    if dtype == "fp32":
        x[130:] *= 1e-32                     # (scales below 2^-90)
    x = x.to(DT[dtype])
    q = torch.empty(150, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-150 // block_rows), -(-cols // 128), device="cuda")
    rs.reshard_fp8_quantize(x, q, s, (150, cols), dtype, block_rows)
    want, _ = oo.quantize(_f64(x)[None], block_rows)
    negative = torch.signbit(x).cpu().numpy()
    assert np.array_equal(q.cpu().numpy(), _bytes(want[0], negative))


# ---------------------------------------------------------------------------- balance
@pytest.mark.parametrize("experts", [1, 8])       # rows off and on 16 bytes
def test_balance_of_nearly_2_31_tokens(experts):
    """Every token of the longest sequence is reached, and none beyond it."""
    n, gone = 2 ** 31 - 8, 3
    logits = torch.zeros(1, n, experts, dtype=torch.float16, device="cuda")
    choices = torch.zeros(1, n, 1, dtype=torch.int32, device="cuda")
    mask = torch.ones(1, n, dtype=torch.uint8, device="cuda")
    mask[0, n - gone:] = 0
    dlogits = torch.empty_like(logits)
    ends = [slice(0, 10 ** 6), slice(n - 10 ** 8, n)]
    for e in ends:
        dlogits[:, e] = 7.0
    counts = torch.empty(1, experts, dtype=torch.int32, device="cuda")
    loss = torch.empty(1, device="cuda")
    shape = (1, n, experts)
    workspace = torch.empty(rs.reshard_balance_loss_workspace(shape), dtype=torch.uint8, device="cuda")
    rs.reshard_balance_loss(logits, shape, "fp16", choices, 1, 1.0, workspace, counts, loss=loss,
                            dlogits=dlogits, mask=mask)
    assert counts[0].tolist() == [n - gone] + [0] * (experts - 1)
    # f = E for the one expert, p = 1 / E: 1 a token; sums of at most 2^18 ones are exact,
    # their shares of n and the loss round three times
    assert abs(float(loss) - 1.0) <= 4 * 2.0 ** -24
    for e in ends:                           # gradients of 2^-31 are 0 in float16
        assert not bool(dlogits[:, e].any())


def _many_sequences(n, experts=16, topk=2):
    g = torch.Generator(device="cuda").manual_seed(n)
    logits = torch.randn(n, 1, experts, generator=g, device="cuda")
    choices = logits.topk(topk, dim=2).indices.to(torch.int32)
    mask = (torch.rand(n, 1, generator=g, device="cuda") < 0.7).to(torch.uint8)
    shape = (n, 1, experts)
    workspace = torch.empty(rs.reshard_balance_loss_workspace(shape), dtype=torch.uint8, device="cuda")
    counts = torch.empty(n, experts, dtype=torch.int32, device="cuda")
    loss, dlogits = torch.empty(1, device="cuda"), torch.full_like(logits, 7.0)

    def call():
        rs.reshard_balance_loss(logits, shape, "fp32", choices, topk, 1.0, workspace, counts, loss=loss,
                                dlogits=dlogits, mask=mask)
    return call, logits, choices, mask, counts, loss, dlogits


@pytest.mark.parametrize("n", [1024, 1025, 300000])
def test_balance_of_many_sequences(n):
    experts, topk = 16, 2
    call, logits, choices, mask, counts, loss, dlogits = _many_sequences(n, experts, topk)
    for _ in range(2):                       # the second call finds the first one's workspace
        call()
    on = mask[:, 0] != 0
    want = torch.zeros(n, experts, dtype=torch.int32, device="cuda")
    want.scatter_(1, choices[:, 0].long(), 1)
    want[~on] = 0
    assert torch.equal(counts, want)
    live = int(on.sum())
    p = torch.softmax(logits[:, 0].double(), dim=1)
    f = want.double() * experts / topk
    dot = (p * f).sum(1, keepdim=True)
    grad = p * (f - dot) / live
    # as for the smaller sizes: E / 32 + 53 roundings, of what is added up
    rel = (experts / 32 + 53) * 2.0 ** -23
    assert abs(float(loss) - float(dot[on].sum()) / live) <= 2 * rel * float(dot[on].sum()) / live
    off = (dlogits[:, 0].double() - grad).abs()
    assert bool((off <= 2 * rel * p * (f + dot) / live)[on].all())
    assert not bool(dlogits[~on].any())


def test_balance_takes_time_in_proportion_to_the_sequences():
    """16 times the sequences take at most three times 16 times as long (256 times as long if
    each sequence looked at all the others)."""
    def us(n):
        call = _many_sequences(n)[0]
        times = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[3]
    assert us(16 * 32768) <= 48 * us(32768)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [40, 3000])    # one launch, and two
@pytest.mark.parametrize("experts", [8, 9, 1100])
def test_balance_scores_far_from_zero(experts, tokens, score):
    """Small scores are as exact, relative to themselves, as large ones."""
    g = torch.Generator(device="cuda").manual_seed(experts)
    if score == "softmax":                   # one likely expert, the others e^-20 to e^-85 of it
        logits = -20 - 65 * torch.rand(1, tokens, experts, generator=g, device="cuda")
        logits[:, :, 3] = 0.0
    else:                                    # none likely
        logits = -80 - 6 * torch.rand(1, tokens, experts, generator=g, device="cuda")
    choices = (torch.arange(tokens, device="cuda") % experts).to(torch.int32).view(1, tokens, 1)
    shape = (1, tokens, experts)
    workspace = torch.empty(rs.reshard_balance_loss_workspace(shape), dtype=torch.uint8, device="cuda")
    counts = torch.empty(1, experts, dtype=torch.int32, device="cuda")
    dlogits = torch.empty_like(logits)
    rs.reshard_balance_loss(logits, shape, "fp32", choices, 1, float(tokens), workspace, counts,
                            dlogits=dlogits, score=score)
    l = logits[0].double()
    f = counts[0].double() * experts / tokens
    if score == "softmax":
        p = torch.softmax(l, dim=1)
        slope = p
    else:
        p = torch.sigmoid(l) / torch.sigmoid(l).sum(1, keepdim=True)
        slope = p * torch.sigmoid(-l)
    dot = (p * f).sum(1, keepdim=True)
    grad = slope * (f - dot)
    # In units of 2^-24: an exponential 4 (2^x) + 4 (t's part of ln 2) + 2 (1 + t, the product), the
    # difference l - top that it is taken of |z| / 2 at most where that is not exact (it is: top
    # is 0); the sigmoid 1 + 2; the sum as much again and E / 32 + 5 additions; 9 for f, its mean
    # (whose own terms are as far off), the quotient and the products.
    each = 4 + 4 + 2 + 3
    rel = (2 * each + 2 * (experts / 32 + 5) + 9) * 2.0 ** -24
    off = (dlogits[0].double() - grad).abs()
    assert bool((off <= rel * slope * (f + dot) + 2.0 ** -126).all()), float(
        (off / (slope * (f + dot)).clamp_min(2.0 ** -100)).max() * 2 ** 24)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [200, 20000])  # one launch, and two
def test_balance_of_a_score_next_to_one(tokens, score):
    """The gradient of an expert whose score is e^-80 to e^-87 next to another one's 1, with all
    choices: f = (0, 2), so that it is 2 p for the score p (in units of coef / n = 1)."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    z = -80 - 7 * torch.rand(tokens, generator=g, device="cuda")
    logits = torch.stack([torch.full_like(z, 0.0 if score == "softmax" else 30.0), z], dim=1)[None]
    choices = torch.ones(1, tokens, 1, dtype=torch.int32, device="cuda")
    shape = (1, tokens, 2)
    workspace = torch.empty(rs.reshard_balance_loss_workspace(shape), dtype=torch.uint8, device="cuda")
    counts = torch.empty(1, 2, dtype=torch.int32, device="cuda")
    dlogits = torch.empty_like(logits)
    rs.reshard_balance_loss(logits, shape, "fp32", choices, 1, float(tokens), workspace, counts,
                            dlogits=dlogits, score=score)
    want = 2 * torch.exp(z.double())
    # In units of 2^-24: 2^x 4, ln 2 in t 4 (|x| 1.9e-9 for |x| <= 126), the correction's product 1, the
    # sigmoid's sum and reciprocal 3; coef / live / n 2, f 3, its product with the share 1, with the
    # score 1, of the sum's reciprocal 2.
    off = ((dlogits[0, :, 1].double() - want) / want).abs().max()
    assert float(off) <= (4 + 4 + 1 + 3 + 2 + 3 + 1 + 1 + 2) * 2.0 ** -24


def test_balance_of_scores_that_are_too_small():
    """Sigmoid scores below 2^-126 are 0: the second token has none."""
    logits = torch.tensor([[[-87.0, -88.0], [-88.0, -90.0]]], device="cuda")
    choices = torch.zeros(1, 2, 1, dtype=torch.int32, device="cuda")
    workspace = torch.empty(rs.reshard_balance_loss_workspace((1, 2, 2)), dtype=torch.uint8, device="cuda")
    counts = torch.empty(1, 2, dtype=torch.int32, device="cuda")
    loss, dlogits = torch.empty(1, device="cuda"), torch.full_like(logits, 7.0)
    rs.reshard_balance_loss(logits, (1, 2, 2), "fp32", choices, 1, 1.0, workspace, counts, loss=loss,
                            dlogits=dlogits, score="sigmoid")
    assert float(loss) == 1.0                # f = (2, 0): 2 of the first token, over two tokens
    assert not bool(dlogits[0, 1].any())


# ----------------------------------------------------------------------------- matmul
@pytest.mark.parametrize("offsets", [[2, 9, 4, 6], [0, 0, 12, 3], [5, 5, 5, 5], [-4, 30, 1, 2], [7, 3, 9, 20]])
def test_matmul_offsets_that_decrease(offsets):
    """An offset below an earlier one counts as that one, with and without an inner size."""
    first, most = min(max(offsets[0], 0), 20), min(max(offsets), 20)
    for k in (0, 16):
        x = torch.full((20, 16), 0x38, dtype=torch.uint8, device="cuda")        # 1.0
        w = torch.full((3, 8, 16), 0x38, dtype=torch.uint8, device="cuda")
        xs, ws = torch.ones(20, 1, device="cuda"), torch.ones(3, 1, 1, device="cuda")
        y = torch.full((20, 8), 77.0, device="cuda")
        rs.reshard_fp8_matmul(x, xs, w, ws, y, (20, 8, k), "fp32",
                              offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                              nexperts=3, ldx=16, ldw=16)
        want = torch.full((20, 8), 77.0)
        want[first:most] = float(k)
        assert torch.equal(y.cpu(), want), k
