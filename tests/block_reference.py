"""Plain 64-bit forms of the block-scaled 8-bit operators, for their tests:
written element by element from the format's definition, on the CPU, sharing no
code with the library."""
from __future__ import annotations

import numpy as np
import torch

import dtensor_layout_movement_amd as R

BLOCK = 128
E4M3, E5M2 = R.DTYPE_FP8_E4M3, R.DTYPE_FP8_E5M2
TOP = {E4M3: 448.0, E5M2: 57344.0}


def decode_table(fmt):
    """The value of every byte of a format, from its bit fields."""
    out = np.empty(256)
    for b in range(256):
        sign = -1.0 if b & 128 else 1.0
        if fmt == E4M3:
            e, m, bits, bias = b >> 3 & 15, b & 7, 3, 7
            special = np.nan if (e == 15 and m == 7) else None
        else:
            e, m, bits, bias = b >> 2 & 31, b & 3, 2, 15
            special = None if e < 31 else (np.inf if m == 0 else np.nan)
        v = special if special is not None else (
            np.ldexp(float(m), 1 - bias - bits) if e == 0 else np.ldexp(float((1 << bits) + m), e - bias - bits))
        out[b] = sign * v
    return out


def round_to_format(v, fmt):
    """Nearest value of the format (ties to even) of finite float64 |v| <= top."""
    bits, low = (3, -6) if fmt == E4M3 else (2, -14)
    _, x = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(x - 1, low) - bits)
    return np.rint(v / step) * step


def quantize(x, block_rows, fmt=E4M3):
    """(values after the round trip, scale bytes) of a 2-d tensor, in float64."""
    x = x.detach().cpu().double().numpy()
    rows, cols = x.shape
    Rb, Cb = -(-rows // block_rows), -(-cols // BLOCK)
    out = np.empty_like(x)
    scales = np.full((Rb, Cb), 127, np.int64)
    for i in range(Rb):
        for j in range(Cb):
            box = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            v = x[box]
            fin = np.isfinite(v)
            amax = np.abs(v[fin]).max() if fin.any() else 0.0
            e = 0
            if amax > 0:
                e = -127
                f, p = np.frexp(amax / TOP[fmt])  # f 2^p with f in [0.5, 1): amax <= top 2^p
                e = max(-127, int(p - 1 if f == 0.5 else p))
                assert amax <= TOP[fmt] * 2.0 ** e and (e == -127 or amax > TOP[fmt] * 2.0 ** (e - 1))
            scales[i, j] = e + 127
            with np.errstate(invalid="ignore"):
                q = np.where(fin, round_to_format(np.where(fin, v, 0.0) / 2.0 ** e, fmt) * 2.0 ** e, np.nan)
            out[box] = q
    return out, scales


def values(payload, scales, rows, cols, block_rows, fmt=E4M3):
    """float64 values of payload and scale bytes (CPU uint8 tensors)."""
    t = decode_table(fmt)
    q = t[payload.cpu().numpy()[:rows, :cols].astype(np.int64)]
    s = scales.cpu().numpy().astype(np.int64)
    u = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    u = np.repeat(np.repeat(u, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]
    return q * u


def rounding(dtype):
    """Half a step of the type relative to a value."""
    return torch.finfo(dtype).eps / 2
