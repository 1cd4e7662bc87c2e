"""Distillation with the teacher's rest as one more outcome, in 64 bits and by logarithms, in numpy, for
one row at a time: no probability underflows, however far the listed tokens lie above the others.

It follows the definition in include/reshard.h and shares nothing with the library.  Bounds count the
definition's float32 steps, as in logit_oracles: an exponent is off by at most 6 roundings of itself, a
power of 2 by 2 units in its last place and, where it is below 2^-126, by all of itself; no term of a
sum over a row of V goes through more than 80 + V / 4096 additions; 1 / T is rounded once; the rest is
off by 2^-41 and a rounding.
"""
import numpy as np

from tests.logit_oracles import U, inverse

FARTHEST = 2.0 ** 15    # T by which all other tokens may lie below the largest logit
FLUSHED = 2.0 ** -126


def distill(x, t, token, y, g, eps):
    """(loss, its bound, gradient, its bound) of one row of cleaned logits with an entry above -inf."""
    V, inv = len(x), inverse(t)
    ok = [(int(i), float(v)) for i, v in zip(token, y) if 0 <= i < V and not np.isnan(v)]
    at, ys = np.array([i for i, _ in ok]), np.array([v for _, v in ok])
    listed = np.zeros(V, bool)
    listed[at] = True
    top = x.max()
    with np.errstate(all="ignore"):
        z = np.where(x == top, 0.0, (x - top) * inv)
    normal = np.log(np.exp(z).sum())
    p = np.exp(z - normal)
    q = np.exp(ys)
    z_rest = z[~listed].max(initial=-np.inf)
    rest = max(0.0, 1.0 - q.sum()) if z_rest >= -FARTHEST else 0.0
    far = z_rest if z_rest > -np.inf else 0.0
    with np.errstate(all="ignore"):
        e = np.where(listed, 0.0, np.exp(z - far))                # others, relative to their largest
    other = e.sum()
    # errors: of an exponential relative to the others' largest, their sum, the way to the top, S
    gap = np.where(e > 0, far - z, 0.0)
    each = 6 * U * gap + 4 * U
    other_off = ((e * each).sum() / other if other > 0 else 0.0) + (80 + V / 4096) * U
    way = 6 * U * abs(far) + 4 * U
    mild = np.where(listed & (z > -200), np.abs(z), 0.0)
    s_off = p[~listed].sum() * (other_off + way) + (p * (6 * U * mild + 4 * U))[listed].sum() + 20 * U
    rest_off = 2.0 ** -41 / rest + U if rest > 0 else 0.0

    zl = z[at]
    loss = np.where(q > 0, q * (ys - (zl - normal)), 0.0).sum()
    loss_off = (q * 1.5 * U * np.abs(zl)).sum() + (q * U * np.abs(ys - zl + normal)).sum() + q.sum() * (s_off + 3 * U)
    slope = g * inv
    grad, off = p * slope, np.zeros(V)
    if rest > 0:
        term = np.log(rest) - (far + np.log(other) - normal)
        loss += rest * term
        loss_off += rest * (rest_off * (abs(term) + 1) + 1.5 * U * abs(far) + other_off + s_off + 6 * U)
        grad = np.where(listed, grad, grad - slope * rest * e / other)
    lead, share = np.exp(far - normal), rest / other if rest > 0 else 0.0
    lead_off = lead * (way + s_off + 4 * U) + share * (rest_off + other_off + 4 * U) + FLUSHED
    off = abs(slope) * (e * lead_off + abs(lead - share) * (e * (each + 6 * U) + FLUSHED))
    for i in np.unique(at):
        mass = q[at == i].sum()
        grad[i] = slope * (p[i] - mass)
        off[i] = abs(slope) * (p[i] * (6 * U * mild[i] + s_off + 10 * U) + FLUSHED + 8 * U * mass)
    return loss, loss_off + U * abs(loss), grad, off + eps[0] * (np.abs(grad) + off) + eps[1]
