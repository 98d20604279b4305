"""The plain implementations of routing and codes hold their own definitions (CPU)."""

import numpy as np
import pytest

from oracle import blocks as B
from oracle import experts as O


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_equals_differences(score, renormalize):
    rng = np.random.default_rng(0)
    z = rng.standard_normal((7, 12))
    z[3, 4] = -np.inf
    chosen, w = O.route(z, 3, score=score, renormalize=renormalize, scale=2.5)
    assert np.allclose(w, O.weights_of(z, chosen, score, renormalize, 2.5), rtol=1e-12)
    g = rng.standard_normal((7, 3))
    got = O.route_backward(z, chosen, g, score, renormalize, 2.5)
    h = 1e-6
    for t in range(7):
        for e in range(12):
            if not np.isfinite(z[t, e]):
                assert got[t, e] == 0
                continue
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            d = ((O.weights_of(up, chosen, score, renormalize, 2.5) -
                  O.weights_of(down, chosen, score, renormalize, 2.5)) * g).sum() / (2 * h)
            assert abs(d - got[t, e]) < 1e-8


def test_ties_masks_and_empty_rows():
    z = np.array([[1.0, 2.0, 2.0, 0.0], [-np.inf] * 4, [np.nan, 0, 0, 0], [-np.inf, 5.0, -np.inf, -np.inf]])
    chosen, w = O.route(z, 2)
    assert chosen.tolist() == [[1, 2], [-1, -1], [-1, -1], [1, -1]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [0, 0] and np.isnan(w[2]).all() and w[3].tolist() == [1, 0]
    chosen, _ = O.route(z, 2, mask=[False, True, True, True])
    assert chosen[0].tolist() == [-1, -1]
    # a bias chooses and does not weigh
    chosen, w = O.route(z[:1], 1, bias=np.array([0, 0, 0, 9.0]), renormalize=False)
    assert chosen[0, 0] == 3 and w[0, 0] == O.scores(z[0], "softmax")[3]


def test_groups():
    z = np.array([[3.0, 0.0, 2.0, 2.0, 0.0, 0.1]])
    # by the sum of two the second group is best, by the best one the first
    two = O.scores(z, "sigmoid")[0]
    assert two[2] + two[3] > two[0] + two[1]
    assert O.route(z, 2, score="sigmoid", groups=3, top_groups=1)[0].tolist() == [[2, 3]]
    assert O.route(z, 2, score="sigmoid", groups=3, top_groups=1, group_best=1)[0].tolist() == [[0, 1]]


def test_order():
    chosen = np.array([[1, 0], [1, -1], [2, 1]])
    slots, pairs, offsets, loads = O.order(chosen, 4, 1)
    assert pairs.tolist() == [1, 0, 2, 5, 4, -1] and offsets.tolist() == [0, 1, 4, 5, 5] and loads.tolist() == [1, 3, 1, 0]
    assert slots.tolist() == [[1, 0], [2, -1], [4, 3]]
    slots, pairs, offsets, _ = O.order(chosen, 4, 4)
    assert offsets.tolist() == [0, 4, 8, 12, 12] and len(pairs) == 20 and slots[2].tolist() == [8, 6]


def test_code_table():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(codes, B.TABLE, equal_nan=True)
