"""The balance loss at sizes that make its kernels go on from one token to the next and count by
several clusters, against float64 on the GPU."""
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests.test_gpu_operators import DT, EPS

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")


def _check_many(x, choices, mask, topk, score, dtype, coef=0.01):
    """As for small sizes, in float64 on the GPU."""
    S, T, E = x.shape
    x = x.to(DT[dtype])
    workspace = torch.empty(rs.reshard_balance_loss_workspace((S, T, E)), dtype=torch.uint8, device="cuda")
    counts = torch.empty(S, E, dtype=torch.int32, device="cuda")
    loss, dlogits = torch.empty(1, device="cuda"), torch.full_like(x, 7.0)
    rs.reshard_balance_loss(x, (S, T, E), dtype, choices, topk, coef, workspace, counts, loss=loss,
                            dlogits=dlogits, mask=mask, score=score)
    on = torch.ones(S, T, dtype=torch.bool, device="cuda") if mask is None else mask != 0
    want = torch.stack([torch.bincount(choices[s][on[s]].flatten().long(), minlength=E) for s in range(S)])
    assert torch.equal(counts.long(), want)
    tokens = on.sum(1)
    live, n = max(1, int((tokens > 0).sum())), tokens.clamp_min(1).double()[:, None, None]
    f = want.double()[:, None] * E / (topk * n)
    l = torch.where(on[..., None], x, 0).double()
    a = torch.softmax(l, 2) if score == "softmax" else torch.sigmoid(l)
    p = a / a.sum(2, keepdim=True)
    slope = p if score == "softmax" else p * torch.sigmoid(-l)
    dot = (p * f).sum(2, keepdim=True)
    total = float((dot / n)[on].sum()) * coef / live
    rel = (E / 32 + 53) * 2.0 ** -23
    assert abs(float(loss) - total) <= 2 * rel * total
    grad = torch.where(on[..., None], coef / (live * n) * slope * (f - dot), 0)
    size = torch.where(on[..., None], coef / (live * n) * slope * (f + f.amax(2, keepdim=True)), 0)
    eps, tiny = EPS[dtype]
    off = (dlogits.double() - grad).abs() - (2 * rel * size + eps * grad.abs() + tiny + 2.0 ** -133)
    assert float(off.max()) <= 0


@pytest.mark.parametrize("S,T,E,topk,dtype,score", [
    (1, 800003, 8, 2, "bf16", "softmax"),    # a token a thread, seven of them one after the other
    (2, 400001, 13, 3, "fp32", "sigmoid"),   # rows off 16 bytes
    (3, 90000, 64, 6, "fp16", "sigmoid"),
    (1, 60000, 256, 8, "bf16", "sigmoid"),   # several clusters count
    (7, 9001, 200, 4, "fp32", "softmax"),
    (1, 20001, 1000, 3, "bf16", "softmax"),  # a token a warp
    (2, 8003, 1001, 3, "fp16", "sigmoid"),
    (2, 9001, 1100, 5, "fp32", "sigmoid"),   # more experts than a warp's registers hold
])
def test_balance_of_many_tokens_a_thread(S, T, E, topk, dtype, score):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn(S, T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    choices = x.topk(topk, dim=2).indices.to(torch.int32)
    _check_many(x, choices, None, topk, score, dtype)
    at = torch.arange(T, device="cuda")
    mask = torch.ones(S, T, dtype=torch.uint8, device="cuda")
    mask[:, T - T // 3:] = 0                 # padding, and gaps of every length up to 20
    mask[0, at % 211 < at // 211 % 20] = 0
    mask[S // 2 + 1:] *= 1 - (at % 2 == 0).to(torch.uint8)
    x[mask == 0] = float("nan")              # what does not count holds anything
    _check_many(x, choices, mask, topk, score, dtype)


def test_balance_counts_of_several_clusters_agree_every_time():
    """One sequence's choices counted by several clusters (sums of whole numbers)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    choices = torch.randint(-1, 300, (1, 100000, 6), generator=g, device="cuda", dtype=torch.int32)
    want = torch.bincount(choices[(choices >= 0) & (choices < 256)].long(), minlength=256)
    workspace = torch.empty(rs.reshard_balance_loss_workspace((1, 100000, 256)), dtype=torch.uint8, device="cuda")
    logits = torch.zeros(1, 100000, 256, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        counts = torch.full((256,), -7, dtype=torch.int32, device="cuda")
        rs.reshard_balance_loss(logits, (1, 100000, 256), "bf16", choices, 6, 1.0, workspace, counts)
        assert torch.equal(counts.long(), want)
