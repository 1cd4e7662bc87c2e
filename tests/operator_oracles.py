"""Plain 64-bit forms of the operators beside a refit, in numpy, for small sizes.

They follow the definitions in include/reshard.h and share nothing with the library.
Bounds returned with a result are derived from the definitions' float32 steps and
hold for any order of summation.
"""
import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_values():
    """The value of every e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    0x7f and 0xff are NaN, there are no infinities."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if (b & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = -v if b >> 7 else v
    return out


def to_e4m3(v):
    """Nearest e4m3 value (halves to the even mantissa), clamped to +-448; NaN stays NaN."""
    v = np.asarray(v, dtype=np.float64)
    c = np.clip(v, -E4M3_MAX, E4M3_MAX)
    step = 2.0 ** (np.maximum(np.frexp(c)[1] - 1, -6) - 3.0)
    return np.clip(np.round(c / step) * step, -E4M3_MAX, E4M3_MAX)


def quantize(x, block_rows):
    """x [n, r, c] float64 holding values of a narrower type -> (values [n, r, c], scales).

    Both divisions are float32's: of two float32 numbers the float64 quotient rounded to
    float32 is the float32 quotient."""
    n, r, c = x.shape
    R, C = -(-r // block_rows), -(-c // 128)
    q, scale = np.empty_like(x), np.empty((n, R, C), dtype=np.float32)
    with np.errstate(all="ignore"):
        for i in range(R):
            for j in range(C):
                s = np.s_[:, i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
                b = np.abs(x[s])
                most = np.where(np.isnan(b), 0.0, b).max(axis=(1, 2))
                sc = np.maximum((most / E4M3_MAX).astype(np.float32), np.float32(2.0 ** -126))
                scale[:, i, j] = sc
                quot = (x[s] / sc.astype(np.float64)[:, None, None]).astype(np.float32)
                q[s] = to_e4m3(quot)
    return q, scale


def matmul(x, xs, w, ws, offsets, out_eps):
    """x [t, k], w [e, n, k] of e4m3 values, scales xs [t, b], ws [e, ceil(n / 128), b], all
    float64 -> (y [t, n] with NaN in rows of no expert, bound on |error|).

    A block's 128 products are exact and are added in four steps of 32 with at least 23
    bits kept below the largest partial sum: 4 * 33 * 2^-23 of the block's sum of
    magnitudes; the scales and the sum over blocks round B + 2 times in float32; y once."""
    t, k = x.shape
    n, blocks = w.shape[1], xs.shape[1]
    y, mag = np.full((t, n), np.nan), np.zeros((t, n))
    for e in range(len(w)):
        a, z = (0, t) if offsets is None else (int(offsets[e]), int(offsets[e + 1]))
        if z <= a:
            continue
        y[a:z] = 0.0
        for b in range(blocks):
            s = np.s_[:, b * 128:(b + 1) * 128]
            sc = xs[a:z, b, None] * np.repeat(ws[e, :, b], 128)[None, :n]
            y[a:z] += (x[a:z][s] @ w[e][s].T) * sc
            mag[a:z] += (np.abs(x[a:z][s]) @ np.abs(w[e][s]).T) * np.abs(sc)
    return y, (132 * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24) * mag + out_eps * np.abs(y)


def sample(x, temperature, top_k, top_p, min_p, u):
    """One row of logits -> (acceptable tokens, logprob of each token or -inf).

    More than one token is acceptable only where float32's exponentials (2 units in the
    last place, and half a unit each for the difference and the product that they are
    taken of, whose effect grows with |z|) leave open on which side of a threshold a
    running sum falls."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    top = x.max() if x.size else -np.inf
    if top == -np.inf:
        return {-1}, None
    greedy = not temperature > 0
    with np.errstate(all="ignore"):
        # differences beyond float32's range have no weight
        gone = (x != top) & ((x - top).astype(np.float32) == -np.inf)
        z = np.where(x == top, 0.0, (x - top) / (1.0 if greedy else float(temperature)))
        z = np.where(gone, -np.inf, z)
        e = np.exp(z)
    logprob = z - np.log(np.sum(e))
    if greedy:
        return {int(np.argmax(x == top))}, logprob
    order = np.lexsort((np.arange(x.size), -x))
    k = int(top_k) if 0 < top_k < x.size else x.size
    order = order[:k]
    # an exponential is off by at most (3 + 2|z|) 2^-24 of itself, and 2^-41 for its weight
    off = np.where(e > 0, e * (3 + 2 * np.minimum(np.abs(z), 200)) * 2.0 ** -23, 0) + 2.0 ** -41
    tokens = set()
    for lean in (-1, 0, 1):              # thresholds a little lower and higher
        kept = order
        if not top_p >= 1:
            cum = np.cumsum(e[order])
            slack = lean * off[order].sum()
            m = int(np.sum(cum - e[order] < max(0.0, float(top_p)) * cum[-1] + slack))
            kept = order[:max(1, m)] if top_p > 0 else order[:1]
        floor = 1.0 if math.isnan(min_p) else min(1.0, float(min_p))
        kept = kept[(e[kept] >= floor - lean * off[kept]) | (kept == order[0])]
        kept = np.sort(kept)
        cum = np.cumsum(e[kept])
        uu = 0.0 if math.isnan(u) else max(0.0, float(u))
        with_weight = kept[e[kept] >= 2.0 ** -41]
        for tilt in (-1, 0, 1):
            if uu >= 1:
                tokens.add(int(with_weight[-1]))
                continue
            target = uu * cum[-1] + tilt * (off[kept].sum() if uu > 0 else 0.0)
            at = int(np.sum(cum <= target))
            tokens.add(int(kept[at]) if at < len(kept) else int(with_weight[-1]))
    return tokens, logprob


def balance(x, experts, mask, topk, score, coef):
    """(loss, counts, gradient, tokens of each sequence) of logits x [s, t, e]."""
    S, T, E = x.shape
    x = x.astype(np.float64)
    mask = np.ones((S, T), bool) if mask is None else mask != 0
    counts = np.zeros((S, E), np.int64)
    grad = np.zeros(x.shape)
    tokens = mask.sum(1)
    live = max(1, int((tokens > 0).sum()))
    loss = 0.0
    for s in range(S):
        n = int(tokens[s])
        if n == 0:
            continue
        for c in experts[s][mask[s]].reshape(-1):
            if 0 <= c < E:
                counts[s, c] += 1
        f = counts[s] * E / (topk * n)
        for t in np.flatnonzero(mask[s]):
            p, slope = scores(x[s, t], score)
            dot = float(p @ f)
            loss += coef / live / n * dot
            grad[s, t] = coef / (live * n) * slope * (f - dot)
    return loss, counts, grad, tokens


def scores(l, score):
    """(scores p of one token, dp_e/dl_e + p_e (p's own slope without the shared sum))."""
    with np.errstate(over="ignore"):
        if l.max() == -np.inf or (score == "sigmoid" and not (1 / (1 + np.exp(-l))).sum() > 0):
            return np.zeros_like(l), np.zeros_like(l)
        if score == "softmax":
            a = np.exp(l - l.max())
            p = a / a.sum()
            return p, p
        a = 1 / (1 + np.exp(-l))
        p = a / a.sum()
        return p, p * (1 / (1 + np.exp(l)))
