"""CPU pins of the 8-bit states' rounding: which random bits two elements of a
group of 16 share, which bits one element's m and r share, that what they do
not share looks independent, and by how much v = r^2 is high."""

import math

import numpy as np
import pytest

from oracle import adamw_multi as OM

N = 1 << 20
SIGMAS = 6  # of a binomial cell; about 4000 cells are looked at, 2e-9 each


def table_is_flat(x, y):
    """Both 3-bit values take each of their 64 pairs as often as chance has it."""
    n = x.size
    count = np.bincount((x * 8 + y).astype(np.int64), minlength=64)
    assert np.all(np.abs(count - n / 64) <= SIGMAS * math.sqrt(n / 64))


def pair(bits, d):
    """The bits of elements i and i + d of every group of 16, for the i that have one."""
    g = bits.reshape(-1, 16)
    return g[:, :16 - d].reshape(-1), g[:, d:].reshape(-1)


@pytest.fixture(scope="module")
def drawn():
    return OM.random_bits(np.arange(N), 1001, 20251)


@pytest.mark.parametrize("d", range(1, 16))
def test_elements_of_a_group(drawn, d):
    m, r = drawn
    m0, m1 = pair(m, d)
    for top in (17, 8, 0):  # leading, middle and last bits of m
        table_is_flat((m0 >> np.uint64(top)) & np.uint64(7), (m1 >> np.uint64(top)) & np.uint64(7))
    r0, r1 = pair(r, d)
    for top in (17, 12, 7):  # the 13 leading bits of r
        table_is_flat((r0 >> np.uint64(top)) & np.uint64(7), (r1 >> np.uint64(top)) & np.uint64(7))
    # below them the bits 4 to 6, of which the first k are shared where 2^k divides the distance
    k = (d & -d).bit_length() - 1
    differ = np.bitwise_or.reduce(r0 ^ r1)
    assert int(differ) & 0x70 == 0x70 & ~(((1 << k) - 1) << 4)


def test_m_and_r_of_one_element(drawn):
    m, r = drawn
    assert np.array_equal(m >> np.uint64(16), r & np.uint64(15))  # m's leading four are r's last
    assert np.array_equal(r >> np.uint64(16), m & np.uint64(15))
    for a in (17, 10, 4):  # the 16 leading bits of each
        for b in (17, 10, 4):
            table_is_flat((m >> np.uint64(a)) & np.uint64(7), (r >> np.uint64(b)) & np.uint64(7))


def test_v_is_high_by_the_variance_of_r():
    """A code's mean is r, so its square is high by the code's variance, and
    the average collects the excess of 1/(1 - beta2) steps.  A step that moves
    r by d (small beside the code step q) rounds with variance q*|d|; for
    Gaussian gradients |d| is (1 - beta2)/2 * r * 0.97 in the mean, so the excess
    is 0.48 * q/r of v: 3 to 6 % for q/r between 1/16 and 1/8, and the blocks'
    scales, which move too, add to it.  2 to 10 % is asked."""
    n, beta2 = 4096, 0.99
    rng = np.random.default_rng(1)
    values = OM.code_value(np.arange(127))
    codes, scales, zeros = np.zeros(n, dtype=np.uint8), np.zeros((n // 256, 2)), np.zeros(n, dtype=np.uint8)
    v, high = np.zeros(n), []
    for t in range(1, 801):
        g = rng.standard_normal(n)
        v = beta2 * v + (1 - beta2) * g * g
        got = OM.adamw8_step(np.zeros(n), g, zeros, codes, scales, t, 0.0, 0.0, beta2, 1e-8, 0.0, seed=5)
        codes, scales = np.searchsorted(values, got["codes_r"]).astype(np.uint8), got["scales"]
        if t > 400 and t % 20 == 0:
            high.append(np.mean((got["codes_r"] * OM.per_block(scales[:, 1], n)) ** 2) / np.mean(v) - 1)
    assert 0.02 <= np.mean(high) <= 0.10
