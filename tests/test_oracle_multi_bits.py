"""CPU pins of how far the 8-bit states' random bits are independent: which
bits two elements of a group of 16 share, which bits one element's m and r
share, and that what they do not share looks independent."""

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
