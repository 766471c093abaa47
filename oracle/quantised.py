"""CPU oracle for the layer over an 8-bit base weight.

TEST INFRASTRUCTURE.  Only the tests may import or call this module; it
shares no code with the library.

Codes are OCP e4m3 (largest value 448, smallest step 2^-9) under one
power-of-two scale per block: the smallest 2^e, e >= -126, that brings the
block's largest magnitude to at most 448.  Everything is float64, where the
scaled values and the rounding are exact.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
QMAX = 448.0


def exponent(amax: float) -> int:
    """Smallest e >= -126 with amax <= 448 * 2^e."""
    e = -126
    while amax > QMAX * 2.0 ** e:
        e += 1
    return e


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to the even code) of |v| <= 448."""
    v = np.asarray(v, np.float64)
    _, ex = np.frexp(v)                              # |v| = m 2^ex, m in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    return np.rint(v / step) * step


def encode_block(b: np.ndarray):
    """Values over the scale, and the scale byte, of one block."""
    if not np.all(np.isfinite(b)):
        return np.full(b.shape, np.nan), 255
    e = exponent(float(np.max(np.abs(b))))
    return round_e4m3(np.asarray(b, np.float64) * 2.0 ** -e), e + 127


def quantise_rows(X):
    """Values over the scale [T][up(d)], scale bytes [T][ceil(d/128)]."""
    T, d = X.shape
    nb = -(-d // BLOCK)
    v, s = np.zeros((T, nb * BLOCK)), np.zeros((T, nb), np.int64)
    for t in range(T):
        for b in range(nb):
            q, s[t, b] = encode_block(X[t, b * BLOCK:(b + 1) * BLOCK])
            v[t, b * BLOCK:b * BLOCK + q.size] = q
    return v, s


def quantise_weight(W):
    """Values over the scale [d_out][up(d_in)], scale bytes of the 128 x 128 blocks."""
    o, i = W.shape
    no, ni = -(-o // BLOCK), -(-i // BLOCK)
    v, s = np.zeros((o, ni * BLOCK)), np.zeros((no, ni), np.int64)
    for a in range(no):
        for b in range(ni):
            q, s[a, b] = encode_block(W[a * BLOCK:(a + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK])
            v[a * BLOCK:a * BLOCK + q.shape[0], b * BLOCK:b * BLOCK + q.shape[1]] = q
    return v, s


def row_values(v, s, d):
    """What the codes of rows stand for, [T][d]."""
    return (v * np.repeat(2.0 ** (s - 127.0), BLOCK, axis=1))[:, :d]


def weight_values(v, s, d_in):
    """What a weight's codes stand for, [d_out][d_in]."""
    f = np.repeat(np.repeat(2.0 ** (s - 127.0), BLOCK, axis=0)[:v.shape[0]], BLOCK, axis=1)
    return (v * f)[:, :d_in]


def block_amax(V):
    """Largest magnitude of every 128 columns of each row, [rows][ceil(d/128)]."""
    d = V.shape[1]
    return np.stack([np.max(np.abs(V[:, b:b + BLOCK]), axis=1) for b in range(0, d, BLOCK)], axis=1)
