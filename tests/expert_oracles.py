"""Plain 64-bit forms of the operators that take tokens to their experts and back, in numpy.

They follow the definitions in include/reshard.h and share nothing with the library.  Bounds
returned with a result are derived from the definitions' float32 steps and hold for any order
of summation within a chain of the stated length.
"""
import numpy as np


def sort(experts, nexperts):
    """(slot [tokens, topk], offsets [nexperts + 1])."""
    flat = experts.reshape(-1)
    slot = np.full(flat.shape, -1, np.int64)
    offsets, place = [0], 0
    for e in range(nexperts):
        for i in np.flatnonzero(flat == e):
            slot[i] = place
            place += 1
        offsets.append(place)
    return slot.reshape(experts.shape), np.array(offsets)


def combine(rows, slot, weight, eps):
    """rows [n, c] float64, slot [t, k], weight [t, k] or None -> (out [t, c], bound on |error|).

    A sum of k products has k roundings, each at most 2^-24 of the sum of magnitudes so far;
    the result is rounded once more."""
    t, k = slot.shape
    out, mag = np.zeros((t, rows.shape[1])), np.zeros((t, rows.shape[1]))
    for j in range(k):
        for i in range(t):
            if 0 <= slot[i, j] < len(rows):
                term = (1.0 if weight is None else weight[i, j]) * rows[slot[i, j]]
                out[i] += term
                mag[i] += np.abs(term)
    err = k * 2.0 ** -24 * mag
    return out, err + eps[0] * (np.abs(out) + err) + eps[1]


def combine_grad(dout, rows, slot, weight, eps):
    """(drows [n, c] with NaN in rows of no choice, its bound, dweight [t, k], its bound).

    A lane adds at most one product in 32 of a row and what it has goes through 16 more sums
    at most, so that no product takes part in more than c / 32 + 24 of them."""
    t, k = slot.shape
    n, c = rows.shape
    drows, dweight, bound = np.full((n, c), np.nan), np.zeros((t, k)), np.zeros((t, k))
    for i in range(t):
        for j in range(k):
            s = slot[i, j]
            if 0 <= s < n:
                drows[s] = (1.0 if weight is None else weight[i, j]) * dout[i]
                dweight[i, j] = dout[i] @ rows[s]
                bound[i, j] = (c / 32 + 24) * 2.0 ** -24 * (np.abs(dout[i]) @ np.abs(rows[s]))
    return drows, (eps[0] + 2.0 ** -23) * np.abs(drows) + eps[1], dweight, bound
