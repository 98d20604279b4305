"""Every form of the block products against fp64 (oracle/blocks.py): the
few-rows kernels with four and eight waves, one and two row tiles, several
passes and several rounds over k; the tiles of 64, 128 and 256 with two and
four stages, for plain products, batches, rows by expert and gradients, with
several k-tiles each.  The sizes are chosen by the launcher's rule, and each
case says which form that is."""

import numpy as np
import pytest
import torch

from oracle import blocks as O
from tests.test_gpu_blocks import check_product, coded, matrix, of

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


def some(n, around=()):
    """Rows that are looked at: the first and last ones, and those around the borders of tiles."""
    at = set(range(min(n, 20))) | set(range(max(n - 20, 0), n))
    for border in (64, 128, 256, n // 256 * 256, n // 128 * 128, *around):
        at |= set(range(max(border - 4, 0), min(border + 4, n)))
    return np.array(sorted(at))


def check_rows(c, va, vb, at, cols, before=None):
    check_product(c[torch.from_numpy(at).cuda()], *O.product(va[at], vb), cols, None if before is None else before[at])


def accumulated(shape):
    base = torch.randn(shape, generator=torch.Generator().manual_seed(7)).cuda()
    return base, base.clone()


PLAIN = [
    # few rows, four waves: 24 blocks of k are two rounds of four waves; one and two row tiles
    (1, 130, 3000), (16, 100, 4000), (17, 130, 3000), (32, 257, 1200),
    # eight waves: 33 and 65 blocks of k
    (1, 300, 4100), (16, 75, 8200), (17, 130, 4100), (32, 48, 8300),
    # tiles of 64: four stages, more k-tiles than stages
    (65, 300, 1500),
    # tiles of 128 with four stages (144 and 192 tiles), 2, 3 and 8 k-tiles
    (1500, 1500, 1000), (1500, 2000, 200), (2000, 1400, 300),
    # tiles of 128 with two stages (289 tiles), 1, 2 and 5 k-tiles
    (2100, 2100, 100), (2100, 2100, 256), (2100, 2100, 600),
    # bf16 results: tiles of 256 (256 of them), 1, 2 and 3 k-tiles
    (4000, 4000, 128), (4000, 4050, 300),
]


@pytest.mark.parametrize("out", [BF16, F32, "add"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", PLAIN)
def test_plain(mx, m, n, k, block_rows, out):
    a, b = coded(mx, m, k, 1, m + n), coded(mx, n, k, block_rows, k)
    va, vb = of(a), of(b)
    if out == "add":
        base, c = accumulated((m, n))
        mx.block_matmul(a, b, out=c, accumulate=True)
        check_rows(c, va, vb, some(m), k, base.double().cpu().numpy())
    else:
        check_rows(mx.block_matmul(a, b, dtype=out), va, vb, some(m), k)


# (rows 20: few rows; 150: tiles of 64; 900 x 1000: 192 tiles of 128; 1200 x 1300: 330)
@pytest.mark.parametrize("m,n,k", [(20, 130, 700), (150, 200, 900), (900, 1000, 400), (1200, 1300, 260)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batches(mx, m, n, k, dtype):
    a, b = coded(mx, m, k, 1, 1, count=3), coded(mx, n, k, 128, 9, count=3)
    c = mx.block_matmul(a, b, dtype=dtype)
    for i in range(3):
        check_rows(c[i], of(a, i), of(b, i), some(m), k)


ROWS = [
    # few rows: 5 to an expert on average and one of 40 (three passes of 16), 10 and one of 60 (two of 32)
    ([40] + [0] * 7, 130, 1500), ([40] + [0] * 7, 130, 4200),
    ([3, 0, 60, 1, 5, 0, 2, 9], 100, 3000), ([3, 0, 60, 1, 5, 0, 2, 9], 100, 4200), ([24, 23], 75, 520),
    # tiles of 64, of 128 with four stages, of 128 with two
    ([100, 0, 33, 1, 64, 65], 130, 900),
    ([150, 128, 1, 0, 300, 257, 90, 129, 64, 200, 150, 150, 150, 150, 150, 150, 150, 150, 150, 151], 500, 640),
    ([150, 128, 1, 0, 300, 257, 90, 129, 64, 200, 150, 150, 150, 150, 150, 150, 150, 150, 150, 151], 900, 400),
    # bf16 results: tiles of 256 (802 rows to an expert)
    ([1500, 700, 0, 1300, 513], 2600, 300),
]


@pytest.mark.parametrize("out", [BF16, F32, "add"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("lengths,n,k", ROWS)
def test_rows_by_expert(mx, lengths, n, k, block_rows, out):
    at = np.concatenate([[0], np.cumsum(lengths)])
    rows = int(at[-1])
    a, b = coded(mx, rows, k, 1, 1), coded(mx, n, k, block_rows, 50, count=len(lengths))
    offsets = torch.from_numpy(at).int().cuda()
    base, c = accumulated((rows, n))
    if out == "add":
        mx.expert_matmul(a, b, offsets, out=c, accumulate=True)
    else:
        c = mx.expert_matmul(a, b, offsets, dtype=out)
    va = of(a)
    for e, length in enumerate(lengths):
        if length:
            part = slice(int(at[e]), int(at[e + 1]))
            check_rows(c[part], va[part], of(b, e), some(length), k,
                       base[part].double().cpu().numpy() if out == "add" else None)


GRADS = [
    # tiles of 64; of 128 with four stages (192 tiles); with two (288): up to six k-tiles
    (96, 200, [300, 0, 129, 512]), (700, 900, [300, 0, 129, 512]), (700, 900, [300, 0, 129, 512, 700, 1]),
    # bf16 results: tiles of 256 (240)
    (2000, 1500, [300, 128, 1, 0, 400]),
]


@pytest.mark.parametrize("align", [128, 1])
@pytest.mark.parametrize("out", [BF16, F32, "add"])
@pytest.mark.parametrize("m,n,lengths", GRADS)
def test_gradients(mx, m, n, lengths, out, align):
    at = np.concatenate([[0], np.cumsum([-(-x // align) * align for x in lengths])])
    rows = int(at[-1]) + 50
    a, b = mx.quantize(matrix(rows, m, F32, 1), order="cols"), mx.quantize(matrix(rows, n, F32, 2), order="cols")
    offsets = torch.from_numpy(at).int().cuda()
    base, c = accumulated((len(lengths), m, n))
    if out == "add":
        mx.expert_grad(a, b, offsets, out=c, accumulate=True)
    else:
        c = mx.expert_grad(a, b, offsets, dtype=out)
    va, vb = np.pad(of(a), ((0, 0), (0, 8))), np.pad(of(b), ((0, 0), (0, 8)))
    for e in range(len(lengths)):
        lo, hi = int(at[e]), int(at[e + 1])
        first, last = lo // 8 * 8, -(-hi // 8) * 8  # whole groups of the instruction's eight products
        inside = (np.arange(first, last) >= lo) & (np.arange(first, last) < hi)
        check_rows(c[e], va[:, first:last] * inside, vb[:, first:last] * inside, some(m), max(hi - lo, 1) + 128,
                   base[e].double().cpu().numpy() if out == "add" else None)


def test_gradients_of_exact_codes_are_exact(mx):
    """Small integers whose transposed blocks have the largest code, so that every code is its value: sums of integers
    below 2^24 lose nothing in fp32, whatever the expert's rows are."""
    g = torch.Generator().manual_seed(3)
    experts, k, tokens = 4, 2, 64
    x = torch.randint(-4, 5, (tokens, 128), generator=g).to(BF16)
    grad = torch.randint(-2, 3, (tokens, 96), generator=g).to(BF16)
    chosen = torch.randn(tokens, experts, generator=g)
    r = mx.route(chosen.cuda(), k, align=128)
    pairs = r.pairs.cpu().numpy()
    at = r.offsets.tolist()
    # one pair of each block of 128 rows carries 448 in every column of both
    marks = [at[e] for e in range(experts) if at[e + 1] > at[e]]
    xs, gs = x.double().numpy()[np.maximum(pairs, 0) // k], grad.double().numpy()[np.maximum(pairs, 0) // k]
    xs[pairs < 0] = gs[pairs < 0] = 0.0
    for m in marks:
        xs[m], gs[m] = 448.0, 0.0
        gs[m + 1], xs[m + 1] = 448.0, 0.0
    at_codes = mx.quantize(torch.from_numpy(xs).to(BF16).cuda(), order="cols")
    gt_codes = mx.quantize(torch.from_numpy(gs).to(BF16).cuda(), order="cols")
    assert np.array_equal(of(at_codes), xs.T) and np.array_equal(of(gt_codes), gs.T)
    got = mx.expert_grad(gt_codes, at_codes, r.offsets).double().cpu().numpy()
    for e in range(experts):
        assert np.array_equal(got[e], gs[at[e]:at[e + 1]].T @ xs[at[e]:at[e + 1]])


def test_gradients_of_weighted_pairs_are_bounded_by_their_own_terms(mx):
    """The sum over the pairs of w grad x, each factor off by half a step of its code's, bounds each element by itself."""
    g = torch.Generator().manual_seed(3)
    experts, k, tokens = 4, 2, 64
    x = torch.randn(tokens, 128, generator=g).to(BF16).cuda()
    grad = torch.randn(tokens, 96, generator=g).to(BF16).cuda()
    r = mx.route(torch.randn(tokens, experts, generator=g).cuda(), k, align=128)
    _, xt = mx.quantize(x, pairs=(r.pairs, k), order="both")
    _, gt = mx.quantize(grad, pairs=r.pairs, weights=r.weights, order="both")
    got = mx.expert_grad(gt, xt, r.offsets).double().cpu().numpy()
    pairs, at = r.pairs.cpu().numpy(), r.offsets.tolist()
    xs = O.gather(x.double().cpu().numpy(), pairs, k)
    gs = O.gather(grad.double().cpu().numpy(), pairs, k, r.weights.double().cpu().numpy())

    def half_steps(values, codes):
        """What a value's code may be off by."""
        unit = O.spread(codes.scales.double().cpu().numpy(), values.T.shape, 1).T
        q = np.abs(values) / np.where(unit > 0, unit, 1)
        return unit * 0.5 * O.step(q) * (1 + 2.0 ** -20) + np.abs(values) * 2.0 ** -22

    dx, dg = half_steps(xs, xt), half_steps(gs, gt)
    for e in range(experts):
        s = slice(at[e], at[e + 1])
        want = gs[s].T @ xs[s]
        tol = dg[s].T @ np.abs(xs[s]) + np.abs(gs[s]).T @ dx[s] + dg[s].T @ dx[s]
        size = (np.abs(gs[s]) + dg[s]).T @ (np.abs(xs[s]) + dx[s])
        tol += size * (at[e + 1] - at[e] + 8) * 2.0 ** -23
        assert np.all(np.abs(got[e] - want) <= tol)
        if at[e + 1] > at[e]:  # and says something: most results are larger than their bound
            assert np.mean(np.abs(want) > tol) > 0.5
