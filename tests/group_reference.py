"""Plain 64-bit forms of the group-scaled 4-bit operators and of tokens sorted by
expert, for their tests: written element by element from the definitions, on the
CPU, sharing no code with the library."""
from __future__ import annotations

import numpy as np

GROUP = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = np.concatenate([VALUES, -VALUES])


def round_to_format(v):
    """Codes (0 to 7) of the values nearest to finite |v| <= 6, ties to the even code."""
    d = np.abs(np.abs(v)[..., None] - VALUES)
    low = d.min(axis=-1, keepdims=True)
    near = d == low  # one code, or two neighbours
    first = near.argmax(axis=-1)
    both = near.sum(axis=-1) == 2
    return np.where(both & (first % 2 == 1), first + 1, first)


def quantize(x):
    """(values after the round trip, scale bytes) of a 2-d tensor, in float64."""
    x = x.detach().cpu().double().numpy()
    rows, cols = x.shape
    G = -(-cols // GROUP)
    out, scales = np.empty_like(x), np.full((rows, G), 127, np.int64)
    for g in range(G):
        v = x[:, g * GROUP:(g + 1) * GROUP]
        with np.errstate(invalid="ignore"):
            amax = np.abs(v).max(axis=1)
        for r in range(rows):
            box = np.s_[r, g * GROUP:(g + 1) * GROUP]
            if not np.isfinite(x[box]).all():
                scales[r, g], out[box] = 255, np.nan
                continue
            e = 0
            if amax[r] > 0:
                f, p = np.frexp(amax[r] / 6.0)  # f 2^p with f in [0.5, 1): amax <= 6 2^p
                e = max(-127, int(p - 1 if f == 0.5 else p))
                assert amax[r] <= 6 * 2.0 ** e and (e == -127 or amax[r] > 6 * 2.0 ** (e - 1))
            scales[r, g] = e + 127
            u = x[box] / 2.0 ** e
            out[box] = np.copysign(VALUES[round_to_format(u)], u) * 2.0 ** e
    return out, scales


def values(payload, scales, rows, cols):
    """float64 values of payload and scale bytes (uint8 tensors)."""
    b = payload.cpu().numpy()[:rows].astype(np.int64)
    codes = np.stack([b & 15, b >> 4], axis=-1).reshape(rows, -1)[:, :cols]
    s = scales.cpu().numpy()[:rows].astype(np.int64)
    u = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return TABLE[codes] * np.repeat(u, GROUP, 1)[:, :cols]


def sort(ids, first, experts):
    """(offsets, positions) of a 2-d array of choices."""
    flat = np.asarray(ids).reshape(-1)
    position = np.full(flat.shape, -1, np.int64)
    offsets = [0]
    for e in range(experts):
        mine = [i for i, v in enumerate(flat) if v == first + e]
        for n, i in enumerate(mine):
            position[i] = offsets[-1] + n
        offsets.append(offsets[-1] + len(mine))
    return np.array(offsets), position.reshape(np.asarray(ids).shape)


def kept(position, n_rows):
    """(token, choice, row) of every choice that has a row."""
    return [(t, j, int(p)) for (t, j), p in np.ndenumerate(position) if 0 <= p < n_rows]


def gather(x, position, rows):
    """rows (float64) with the tokens' rows put in."""
    out = rows.copy()
    for t, j, p in kept(position, len(rows)):
        out[p] = x[t]
    return out


def combine(rows, position, weights):
    """(sum, sum of the terms' magnitudes) for each token."""
    out = np.zeros((position.shape[0], rows.shape[1]))
    mass = np.zeros_like(out)
    for t, j, p in kept(position, len(rows)):
        term = rows[p] * (1.0 if weights is None else weights[t, j])
        out[t] += term
        mass[t] += np.abs(term)
    return out, mass


def combine_grad(dout, rows, position, weights, drows):
    """(gradient rows put into drows, gradient of the weights, its terms' magnitudes)."""
    drows, dw = drows.copy(), np.zeros(position.shape)
    mass = np.zeros(position.shape)
    for t, j, p in kept(position, len(rows)):
        drows[p] = dout[t] * (1.0 if weights is None else weights[t, j])
        dw[t, j] = (dout[t] * rows[p]).sum()
        mass[t, j] = np.abs(dout[t] * rows[p]).sum()
    return drows, dw, mass
