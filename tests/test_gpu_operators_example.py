"""The example of a refit and a generation step (examples/rollout_step.py) against float64:
the experts' products within the 8-bit format's error, everything else exactly or to
float32."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "rollout_step.py")


def test_rollout_step():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    spec = importlib.util.spec_from_file_location("rollout_step", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out = ex.main(seed=3)
    torch.cuda.synchronize()
    choices = out["choices"].long()
    assert torch.equal(out["counts"].long(), torch.bincount(choices.flatten(), minlength=ex.EXPERTS))
    # the layer in float64
    w, x = out["weights"].double(), out["x"].double()
    for j in range(ex.TOPK):
        want = torch.einsum("th,tfh->tf", x, w[choices[:, j]])
        got = out["y"][:, j].double()
        # e4m3 rounds each factor by at most 2^-4 of itself (or of the block's smallest step),
        # independent of the others: sums of k products are off by about 2 * 2^-4 / sqrt(3) of
        # their root mean square; 1.5 times that bounds the whole
        assert float((got - want).norm() / want.norm()) < 1.5 * 2 * 2.0 ** -4 / 3 ** 0.5
    # the loss and its gradient
    logits = out["router_logits"].double().requires_grad_()
    f = out["counts"].double() * ex.EXPERTS / (ex.TOPK * ex.TOKENS)
    loss = 0.01 * (torch.softmax(logits, 1) * f).sum(1).mean()
    loss.backward()
    assert abs(float(out["loss"]) - float(loss)) <= 1e-5 * float(loss)
    assert float((out["grad"].double() - logits.grad).norm() / logits.grad.norm()) <= 1e-5
    # the draws: inside the vocabulary, with the log-probability of the whole distribution
    lp = torch.log_softmax(out["logits"].double() / 0.8, 1)
    token = out["token"].long()
    assert bool(((token >= 0) & (token < ex.VOCAB)).all())
    want = lp.gather(1, token[:, None])[:, 0]
    assert float((out["logprob"].double() - want).abs().max()) <= 1e-4
