"""Plain fp64 CPU oracle for the many-tensor operators: the gradient norm with
its clip factor, and one AdamW step with 8-bit moments (the 32-bit step is
oracle/adamw.py's, given the scaled gradient).

TEST INFRASTRUCTURE, NOT PRODUCT CODE.  Only the test suite may import this;
the GPU library shares no code with it.

The update is "LLM Optimizers: From SGD and AdamW to SOAP, Muon, and Scalable
Training", sections 5 and 6.  The 8-bit format is the library's own
(include/muon355.h): m and r = sqrt(v) as e4m3 codes with a scale for each
256 elements, rounded stochastically by 20 random bits.  Everything is NumPy
float64 or integers, written from that definition.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 256
TOP = 448.0
LEAST = 2.0 ** -9
TINY = 2.0 ** -100
WORD = (1 << 32) - 1


def grad_norm(grads, max_norm: float):
    """(norm, scale) of a list of arrays."""
    norm = math.sqrt(math.fsum(float(np.sum(np.asarray(g, dtype=np.float64) ** 2)) for g in grads))
    return norm, 1.0 if norm <= max_norm else max_norm / norm


def mix(x):
    x = np.asarray(x, dtype=np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(WORD)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0x9E3779B9)) & np.uint64(WORD)
    return x ^ (x >> np.uint64(16))


def random_bits(positions, step: int, seed: int):
    """20 random bits for m and 20 for r of the elements at these positions."""
    pos = np.asarray(positions, dtype=np.uint64)
    key = mix(mix(np.uint64(step & WORD)) ^ np.uint64(seed))
    group = (pos >> np.uint64(4)) & np.uint64(WORD)
    a = mix(group ^ key)
    b = mix((a + np.uint64(0x6A09E667)) & np.uint64(WORD))
    s = (a + (pos & np.uint64(15)) * b) & np.uint64(WORD)
    rot = ((s << np.uint64(16)) & np.uint64(WORD)) | (s >> np.uint64(16))
    return s >> np.uint64(12), rot >> np.uint64(12)


def round_code(a, bits):
    """The e4m3 value that the magnitude a (at most 448) becomes: floor(a/q + u) * q."""
    a = np.asarray(a, dtype=np.float64)
    e = np.frexp(a)[1] - 1
    q = np.ldexp(1.0, np.maximum(e, -6) - 3)
    return np.floor(a / q + np.asarray(bits, dtype=np.float64) / 2 ** 20) * q


def code_value(codes):
    """The value of e4m3 codes given as uint8."""
    c = np.asarray(codes, dtype=np.int64)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, np.ldexp(f.astype(np.float64), -9), np.ldexp(8.0 + f, e - 10))
    v = np.where((e == 15) & (f == 7), np.nan, v)
    return np.where(c & 0x80, -v, v)


def per_block(x, n):
    """A value per block, spread over its elements."""
    return np.repeat(np.asarray(x, dtype=np.float64), BLOCK)[:n]


def block_scales(x):
    """The scale of each block of x: its largest magnitude / 448."""
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK)
    pad[:n] = np.abs(x)
    top = pad.reshape(-1, BLOCK).max(1)
    return np.where(top < TINY, 0.0, top / TOP)


def scaled(x, scales, least: float):
    """The magnitudes that are rounded to codes."""
    s = per_block(scales, x.size)
    y = np.abs(x) / np.where(s == 0, np.inf, s)
    return np.where(y == 0, 0.0, np.clip(y, least, TOP))


def adamw8_step(param, grad, codes_m, codes_r, scales, step: int, lr: float, beta1: float, beta2: float, eps: float,
                weight_decay: float, scale: float = 1.0, counter: int = 0, seed: int = 0):
    """One step for one tensor (flat arrays; scales [blocks, 2]).  Returns a
    dict: the new parameter, m, r and scales, and the code values."""
    n = param.size
    g = np.asarray(grad, dtype=np.float64) * scale
    m = code_value(codes_m) * per_block(scales[:, 0], n)
    v = (code_value(codes_r) * per_block(scales[:, 1], n)) ** 2
    m1 = beta1 * m + (1.0 - beta1) * g
    v1 = beta2 * v + (1.0 - beta2) * g * g
    r1 = np.sqrt(v1)
    m_hat, v_hat = m1 / (1.0 - beta1 ** step), v1 / (1.0 - beta2 ** step)
    p = (1.0 - lr * weight_decay) * np.asarray(param, dtype=np.float64) - lr * m_hat / (np.sqrt(v_hat) + eps)
    sm, sr = block_scales(m1), block_scales(r1)
    bm, br = random_bits(counter + np.arange(n), step, seed)
    cm = np.sign(m1) * round_code(scaled(m1, sm, 0.0), bm)
    cr = round_code(scaled(r1, sr, LEAST), br)
    return {"param": p, "m": m1, "r": r1, "scales": np.stack([sm, sr], 1), "codes_m": cm, "codes_r": cr,
            "bits_m": bm, "bits_r": br, "m_parts": np.abs(beta1 * m) + np.abs((1.0 - beta1) * g)}
