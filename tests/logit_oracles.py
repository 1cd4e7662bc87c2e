"""Plain 64-bit forms of the operators on rows of logits that train and score, in numpy, for one
row at a time.

They follow the definitions in include/reshard.h and share nothing with the library.  Bounds
returned with a result are derived from the definitions' float32 steps: a difference, a product
with 1 / T and a product with log2(e) / T put an exponent off by at most 6 roundings of itself, a
power of 2 is off by 2 units in its last place, and no term of a sum over a row of V goes through
more than 80 + V / 4096 additions.
"""
import numpy as np

U = 2.0 ** -24     # half a unit in the last place of a float32 near 1
LARGEST = {"bf16": 3.3895313892515355e38, "fp16": 65504.0, "fp32": 3.4028234663852886e38}


def cleaned(x, dtype):
    """Logits as they count: NaN as -inf, +inf as the largest finite value."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    return np.minimum(x, LARGEST[dtype])


def inverse(t):
    t = float(t)
    return min(1 / t, LARGEST["fp32"]) if t > 0 else 1.0


def softmax(x, t):
    """(z, p, ln S, relative error of S and of each p) of cleaned logits; p is 0 where all are -inf."""
    top = x.max()
    if top == -np.inf:
        return np.full(x.shape, -np.inf), np.zeros(x.shape), 0.0, 0.0, np.zeros(x.shape)
    with np.errstate(all="ignore"):
        z = np.where(x == top, 0.0, (x - top) * inverse(t))
        e = np.exp(z)
    s = e.sum()
    p = e / s
    mild = np.where(p > 0, np.maximum(z, -800), 0.0)
    each = 6 * U * np.abs(mild) + 4 * U
    off = (p * each).sum() + (80 + len(x) / 4096) * U
    return z, p, np.log(s), off, each + off + 4 * U


def logprob(x, t, target):
    """(value, bound); nothing else than -inf for a token without probability."""
    z, p, normal, off, _ = softmax(x, t)
    if x.max() == -np.inf or x[target] == -np.inf:
        return -np.inf, 0.0
    v = z[target] - normal
    if v <= -2.0 ** 128 * (1 - 2.0 ** -25):   # half a step beyond float32's largest rounds to -inf
        return -np.inf, 0.0
    return v, 6 * U * abs(z[target]) + off + 4 * U * normal + U * abs(v)


def entropy(x, t):
    z, p, normal, off, each = softmax(x, t)
    if x.max() == -np.inf:
        return 0.0, 0.0
    mild = np.where(p > 0, z, 0.0)
    v = normal - (p * mild).sum()
    mean = (p * np.abs(mild)).sum()
    bound = off + 4 * U * normal + (p * np.abs(mild) * (each + off)).sum() + (100 + len(x) / 4096) * U * mean
    return v, bound + U * abs(v)


def most_likely(x, k):
    """The k largest logits' tokens, ties to the lowest index, -1 where there are no more."""
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf][:k]
    return np.concatenate([order, np.full(k - len(order), -1)]).astype(np.int64)


def logprob_grad(x, t, target, g, h, eps):
    """(gradient, bound) for the gradients g of the log-probability and h of the entropy."""
    z, p, normal, off, each = softmax(x, t)
    if x.max() == -np.inf:
        return np.zeros(x.shape), np.zeros(x.shape)
    H, Hoff = entropy(x, t)
    inv = inverse(t)
    mild = np.where(p > 0, z, 0.0)
    one = np.zeros(x.shape)
    one[target] = 1.0
    inner = mild - normal + H
    v = inv * (g * (one - p) - h * p * inner)
    wide = np.abs(mild) + normal + H   # terms that cancel in inner
    err = inv * (abs(g) * (p * (each + 8 * U) + one * 4 * U)
                 + abs(h) * p * (np.abs(inner) * (each + 8 * U) + 8 * U * wide + off + Hoff + 6 * U * np.abs(mild)))
    err += 4 * U * inv * abs(g) * p   # A is one sum of both
    return v, err + eps[0] * (np.abs(v) + err) + eps[1]


def distill(x, t, token, y, tail, g, eps):
    """(loss, its bound, gradient, its bound) of one row; loss and gradient 0 for a row that does not
    count.  The list's part is in 64 bits but for q (4 units where it is scaled to 1); ln S is off by
    what S is."""
    V = len(x)
    ok = [(int(i), float(v)) for i, v in zip(token, y) if 0 <= i < V and not np.isnan(v)]
    if not any(v > -np.inf for _, v in ok):
        return 0.0, 0.0, np.zeros(V), np.zeros(V)
    if x.max() == -np.inf:
        return np.inf, 0.0, np.zeros(V), np.zeros(V)
    z, p, normal, off, each = softmax(x, t)
    ys = np.array([v for _, v in ok])
    at = np.array([i for i, _ in ok])
    inside = np.zeros(V, bool)
    inside[at] = True
    p_rest = p[~inside].sum()
    if tail:
        q, log_q, rest, q_off = np.exp(ys), ys, 0.0, 0.0
        rest = max(0.0, 1.0 - q.sum()) if p_rest > 0 else 0.0
    else:
        log_q = ys - ys.max()
        log_q = log_q - np.log(np.exp(log_q).sum())
        # a float32 exponential of a float32 difference
        q, rest, q_off = np.exp(log_q), 0.0, 8 * U * (2 + np.abs(np.where(ys > -np.inf, ys - ys.max(), 0)).max())
    with np.errstate(all="ignore"):
        terms = np.where(q > 0, q * (log_q - (z[at] - normal)), 0.0)
    loss = terms.sum() + (rest * np.log(rest / p_rest) if rest > 0 else 0.0)
    mass = q.sum() + rest
    size = np.where(q > 0, q * (np.abs(np.where(q > 0, log_q, 0)) + np.abs(np.where(np.isfinite(z[at]), z[at], 0))
                                + normal + 1), 0.0).sum()
    loss_off = 3 * off * mass + (q * 4 * U * np.abs(np.where(np.isfinite(z[at]), z[at], 0))).sum() + 2 * q_off * size
    share = rest / p_rest if rest > 0 else 0.0
    grad = p * (1 - share)
    grad_off = p * ((each + 8 * U) * abs(1 - share) + share * (2 * off + 8 * U) + 2 * U)
    for i, v in zip(at, q):
        if inside[i]:
            grad[i] = p[i]
            inside[i] = False
            grad_off[i] = p[i] * (each[i] + 8 * U)
        grad[i] -= v
        grad_off[i] += v * (q_off + 4 * U)
    f = g * inverse(t)
    grad, grad_off = grad * f, grad_off * abs(f) + 4 * U * np.abs(grad * f)
    return loss, loss_off + U * abs(loss), grad, grad_off + eps[0] * (np.abs(grad) + grad_off) + eps[1]
