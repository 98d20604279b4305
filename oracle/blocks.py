"""Plain fp64 implementations of the 8-bit block codes and of their products
(CPU, numpy; test infrastructure only, no code shared with the library)."""

import numpy as np

BLOCK = 128
TOP = 448.0
TINY = 2.0 ** -100


def e4m3_table():
    """The value of every e4m3 code (OCP: bias 7, no infinity, 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        out[c] = np.nan if c & 127 == 127 else s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return out


TABLE = e4m3_table()


def step(y):
    """Distance of neighbouring codes at |y|."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    return 2.0 ** (e - 3)


def tops(x, block_rows):
    """Largest magnitude of every block: [blocks of columns, blocks of rows]."""
    rows, cols = x.shape
    out = np.zeros((-(-cols // BLOCK), -(-rows // block_rows)))
    for c in range(out.shape[0]):
        for r in range(out.shape[1]):
            out[c, r] = np.abs(x[r * block_rows:(r + 1) * block_rows, c * BLOCK:(c + 1) * BLOCK]).max(initial=0.0)
    return out


def spread(s, shape, block_rows):
    """A value for each block, over the block's elements."""
    return np.repeat(np.repeat(s.T, block_rows, 0)[:shape[0]], BLOCK, 1)[:, :shape[1]]


def values(codes, scales, block_rows):
    """codes: uint8 [rows, cols]."""
    return TABLE[codes] * spread(scales.astype(np.float64), codes.shape, block_rows)


def gather(x, pairs, k, weights=None):
    """Rows pairs // k of x, times their weights; zeros where a pair is negative or behind x."""
    out = np.zeros((len(pairs), x.shape[1]))
    for i, p in enumerate(pairs):
        if 0 <= p and p // k < x.shape[0]:
            out[i] = x[p // k] * (1.0 if weights is None else weights.reshape(-1)[p])
    return out


def product(a, b):
    """(A B^T, the sums of magnitudes |A| |B|^T, what the matrix instruction may drop).

    The instruction for 8-bit floats adds eight neighbouring products at a time, after it has cut each off 13 bits
    below the leading bit of the largest one's exponents: of a product 2^-13 of the largest everything remains, of
    one 2^-14 of it nothing does.  So each of the eight loses less than 2^-13 of the largest.
    """
    cols = a.shape[1]
    lost = np.zeros((a.shape[0], b.shape[0]))
    for k in range(0, cols, 8):
        most = np.zeros_like(lost)
        for j in range(k, min(cols, k + 8)):
            np.maximum(most, np.abs(np.outer(a[:, j], b[:, j])), out=most)
        lost += most
    return a @ b.T, np.abs(a) @ np.abs(b).T, lost * 8 * 2.0 ** -13
