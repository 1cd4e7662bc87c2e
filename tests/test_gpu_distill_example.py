"""The example of a training step on a rollout (examples/distill_step.py): its losses and every
gradient against automatic differentiation in float64 of the same step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "distill_step.py")


def test_distill_step():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    spec = importlib.util.spec_from_file_location("distill_step", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out = ex.main(seed=4)
    torch.cuda.synchronize()
    leaves = {k: out[k].double().requires_grad_() for k in ("x", "weights", "head", "gate")}
    x, w, head, gate = leaves.values()
    choices = out["choices"].long()
    y = torch.einsum("th,tkfh->tkf", x, w[choices])
    z = ((y * gate[..., None]).sum(1) @ head) / out["temperature"].double()[:, None]
    logp = torch.log_softmax(z, 1)
    p, q = logp.exp(), out["logprob"].double().exp()
    at = out["token"].long()
    # the teacher's list is of its own logits, in order, at the temperature
    want = torch.log_softmax(out["teacher"].double() / out["temperature"].double()[:, None], 1).topk(ex.LISTED, dim=1)
    assert torch.equal(want.indices, at)
    assert float((want.values - out["logprob"].double()).abs().max()) <= 1e-5
    rest, p_rest = 1 - q.sum(1), 1 - p.gather(1, at).sum(1)
    divergence = (q * (q.log() - logp.gather(1, at))).sum(1) + rest * (rest / p_rest).log()
    score = logp.gather(1, out["drawn"].long()[:, None])[:, 0]
    entropy = -(p * logp).sum(1)
    total = divergence.sum() - (out["advantage"].double() * score).sum() - out["bonus"] * entropy.sum()
    total.backward()
    # float32 products of 256 to 384 terms in cuBLAS and in the kernels: 384 roundings of 2^-24 at most
    bound = 384 * 2.0 ** -24
    for got, ref in ((out["divergence"], divergence), (out["score"], score), (out["entropy"], entropy)):
        assert float((got.double() - ref).norm()) <= 4 * bound * float(ref.norm())
    for name in leaves:
        got, ref = out["d" + name].double(), leaves[name].grad
        assert float((got - ref).norm()) <= 16 * bound * float(ref.norm()), name
