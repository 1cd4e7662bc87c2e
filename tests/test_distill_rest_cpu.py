"""The oracle of distillation with the teacher's rest, without a GPU: against differences of its loss, against
the plain 64-bit form where that does not underflow, and where all mass of the student is on the list."""
import numpy as np
import pytest

from tests import logit_oracles as lo
from tests import rest_oracles as ro

TOKEN, Y = np.array([3, 9, 3, 29, -1]), np.log(np.array([0.3, 0.2, 0.1, 0.15, 0.1]))


def _row(gap, t):
    """30 logits whose listed tokens lie about gap * t above the others."""
    x = np.random.default_rng(3).normal(size=30) * t
    x[[3, 9, 29]] += gap * t
    return x


@pytest.mark.parametrize("t", [0.01, 0.7, 2.0])
@pytest.mark.parametrize("gap", [0, 30, 90, 2000])
def test_gradient_against_differences(gap, t):
    x = _row(gap, t)
    loss = lambda a: ro.distill(a, t, TOKEN, Y, 1.0, (0.0, 0.0))[0]  # noqa: E731
    grad = ro.distill(x, t, TOKEN, Y, 1.0, (0.0, 0.0))[2]
    assert abs(grad.sum()) * t < 1e-12
    for i in range(30):
        step = np.zeros(30)
        step[i] = 1e-4 * t
        assert abs((loss(x + step) - loss(x - step)) / 2e-4 - grad[i] * t) < 1e-7


@pytest.mark.parametrize("gap", [0, 30, 80, 600])
def test_as_the_plain_form(gap):
    x = _row(gap, 0.7)
    a, b = ro.distill(x, 0.7, TOKEN, Y, 1.3, (0.0, 0.0)), lo.distill(x, 0.7, TOKEN, Y, True, 1.3, (0.0, 0.0))
    assert abs(a[0] - b[0]) < 1e-11 and np.all(np.abs(a[2] - b[2]) < 1e-12)


def test_the_rest_has_nowhere_to_be():
    for low in (-np.inf, -lo.LARGEST["fp32"], -lo.LARGEST["fp16"]):
        x = np.full(30, low)
        x[[3, 9, 29]] = 0.0
        a, b = ro.distill(x, 0.7, TOKEN, Y, 1.0, (0.0, 0.0)), lo.distill(x, 0.7, TOKEN, Y, True, 1.0, (0.0, 0.0))
        assert abs(a[0] - b[0]) < 1e-11 and np.all(np.abs(a[2] - b[2]) < 1e-12)
