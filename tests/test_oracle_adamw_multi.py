"""CPU pins of the many-tensor oracle: the e4m3 values against torch's
float8_e4m3fn, the stochastic rounding's bounds and expectation, the random
bits, and the limits in which the 8-bit step must be the plain AdamW step."""

import math

import numpy as np
import pytest
import torch

from oracle import adamw as OA
from oracle import adamw_multi as OM


def test_code_values_are_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(OM.code_value(codes.numpy()), want, equal_nan=True)


def test_rounding_gives_neighbours_and_keeps_codes():
    values = np.unique(np.abs(OM.code_value(np.arange(127))))
    rng = np.random.default_rng(0)
    bits = rng.integers(0, 1 << 20, values.size)
    assert np.array_equal(OM.round_code(values, bits), values)  # a code is itself for every u
    x = np.exp(rng.uniform(math.log(2.0 ** -12), math.log(448.0), 20000))
    u = rng.integers(0, 1 << 20, x.size)
    got = OM.round_code(x, u)
    at = np.searchsorted(values, x, side="right") - 1
    low, high = values[at], values[np.minimum(at + 1, values.size - 1)]
    assert np.all((got == low) | (got == high))
    assert np.array_equal(OM.round_code(x, np.zeros_like(u)), low)


def test_rounding_is_unbiased():
    # all 2^20 values of u: the mean is y to the spacing of u
    u = np.arange(1 << 20)
    for y in (0.0007, 0.013, 0.3, 1.0, 5.37, 447.3):
        mean = float(np.mean(OM.round_code(np.full(u.size, y), u)))
        q = 2.0 ** (max(math.floor(math.log2(y)), -6) - 3)
        assert abs(mean - y) <= q * 2.0 ** -20


def test_random_bits_are_uniform_and_differ_by_seed_and_step():
    pos = np.arange(1 << 18)
    m, r = OM.random_bits(pos, 7, 3)
    n = pos.size
    for b in (m, r):
        b = b.astype(np.float64) / 2 ** 20
        # mean of n uniforms: 1/2 +- 5 sigma, sigma = 1/sqrt(12 n); second moment likewise
        assert abs(b.mean() - 0.5) <= 5 / math.sqrt(12 * n)
        assert abs((b ** 2).mean() - 1 / 3) <= 5 * math.sqrt(4 / 45 / n)
        # each of 64 bins: n/64 +- 5 sqrt(n/64)
        hist = np.histogram(b, 64, (0.0, 1.0))[0]
        assert np.all(np.abs(hist - n / 64) <= 5 * math.sqrt(n / 64))
    corr = np.corrcoef(m.astype(np.float64), r.astype(np.float64))[0, 1]
    assert abs(corr) <= 5 / math.sqrt(n)
    # neighbours in position
    assert abs(np.corrcoef(m[1:].astype(float), m[:-1].astype(float))[0, 1]) <= 5 / math.sqrt(n)
    for other in (OM.random_bits(pos, 8, 3), OM.random_bits(pos, 7, 4)):
        assert np.mean(other[0] == m) < 1e-3


def test_grad_norm_closed_forms():
    assert OM.grad_norm([np.full(4, 3.0)], 12.0) == (6.0, 1.0)
    assert OM.grad_norm([np.array([3.0]), np.array([[4.0]])], 1.0) == (5.0, 0.2)
    assert OM.grad_norm([np.zeros(3)], 1.0) == (0.0, 1.0)
    assert OM.grad_norm([np.array([3e38])], math.inf)[0] == pytest.approx(3e38)  # over fp32's range when squared


def test_first_step_is_adamw():
    """From zero states the 8-bit step's parameter is the plain AdamW step's
    exactly, and its moments are, before rounding."""
    rng = np.random.default_rng(1)
    n = 700
    p, g = rng.standard_normal(n), rng.standard_normal(n)
    z = np.zeros(n, dtype=np.uint8)
    got = OM.adamw8_step(p, g, z, z, np.zeros((3, 2)), 1, 1e-2, 0.9, 0.999, 1e-8, 0.1)
    want = OA.adamw_step(p, g, np.zeros(n), np.zeros(n), 1, 1e-2, 0.9, 0.999, 1e-8, 0.1)
    for a, b in zip((got["param"], got["m"], got["r"] ** 2), want):
        assert np.allclose(a, b, rtol=1e-12, atol=0)
    # dequantized moments lie within one code step: at most 1/8 of the value, or 2^-9 scales
    sm = OM.per_block(got["scales"][:, 0], n)
    assert np.all(np.abs(got["codes_m"] * sm - got["m"]) <= np.maximum(np.abs(got["m"]) / 8, sm * 2.0 ** -9))


def test_small_r_keeps_a_code_and_zero_stays_zero():
    n = 256
    g = np.full(n, 1e-9)
    g[0], g[1] = 1.0, 0.0
    z = np.zeros(n, dtype=np.uint8)
    got = OM.adamw8_step(np.zeros(n), g, z, z, np.zeros((1, 2)), 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
    assert got["codes_r"][0] == 448.0 and got["codes_r"][1] == 0.0 and got["codes_m"][1] == 0.0
    assert np.all(got["codes_r"][2:] == 2.0 ** -9)
    tiny = OM.adamw8_step(np.zeros(n), np.full(n, 1e-32), z, z, np.zeros((1, 2)), 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
    assert np.all(tiny["scales"] == 0.0) and np.all(tiny["codes_r"] == 0.0)


def test_average_follows_a_falling_gradient():
    """What round-to-nearest cannot do: r decays after the gradient falls, and
    its mean follows the exact average.  Per step a code's variance is at most
    q * |change| and the average forgets with 1 - beta2, so the mean square of
    the 4096 elements stays within a few per cent: 10 % is asked, where a
    stalled average would be off by more than 600 %."""
    n, beta2 = 4096, 0.99
    codes, scales = np.zeros(n, dtype=np.uint8), np.zeros((n // 256, 2))
    table = {float(v): c for c, v in enumerate(OM.code_value(np.arange(127)))}
    v = 0.0
    for t in range(1, 401):
        g = 1.0 if t <= 100 else 0.05
        v = beta2 * v + (1 - beta2) * g * g
        got = OM.adamw8_step(np.zeros(n), np.full(n, g), np.zeros(n, dtype=np.uint8), codes, scales, t, 0.0, 0.0, beta2,
                             1e-8, 0.0, seed=5)
        codes = np.array([table[float(x)] for x in got["codes_r"]], dtype=np.uint8)
        scales = got["scales"]
    mean = np.mean((got["codes_r"] * OM.per_block(scales[:, 1], n)) ** 2)
    assert abs(mean / v - 1) <= 0.1
