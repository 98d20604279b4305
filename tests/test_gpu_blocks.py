"""GPU parity of the 8-bit block codes and their products with plain fp64
implementations (oracle/blocks.py): odd sizes, strides, both orders, gathered
rows, batches, experts without rows, refusals, graphs and streams."""

import math

import numpy as np
import pytest
import torch

from oracle import blocks as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


def matrix(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2.0 * torch.randn(rows, 1, generator=g))
    x *= torch.exp(torch.randn(1, cols, generator=g))
    x[torch.rand(rows, generator=g) < 0.1] = 0.0
    return x.to(dtype).cuda()


def raw(codes):
    """The code bytes on the host."""
    return codes.contiguous().view(torch.uint8).cpu().numpy()


def padding(q):
    """The codes behind the last column."""
    wide = -(-q.cols // 128) * 128
    size = (*q.codes.shape[:-1], wide)
    return raw(q.codes.as_strided(size, q.codes.stride()))[..., q.cols:]


def check_codes(q, x, block_rows):
    """Codes q of the fp64 matrix x: the scale is the correctly rounded quotient, a value is off by half a step.

    The quotient is within 2^-23 of itself before it is rounded (its correction leaves half a unit in the last
    place of fp32, and so does 0.875 x for fp32 inputs): where it lies that near to half-way between two codes,
    either of them is right."""
    top = O.tops(x, block_rows)
    top[top < O.TINY] = 0.0
    scale = q.scales.cpu().numpy()
    assert np.array_equal(scale, (top.astype(np.float32) / np.float32(448.0)))
    got = O.TABLE[raw(q.codes)]
    most = O.spread(top, x.shape, block_rows)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where(most > 0, 448.0 * x / most, 0.0)
    assert np.all(np.abs(got - y) <= 0.5 * O.step(y) + np.abs(y) * 2.0 ** -22)
    assert not padding(q).any()


SHAPES = [(1, 1), (1, 128), (3, 127), (16, 129), (17, 640), (128, 128), (129, 255), (300, 1000), (1000, 130)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_of_both_orders(mx, rows, cols, block_rows, dtype):
    x = matrix(rows, cols, dtype, rows + cols)
    ref = x.double().cpu().numpy()
    q, qt = mx.quantize(x, block_rows=block_rows, order="both")
    check_codes(q, ref, block_rows)
    check_codes(qt, ref.T, block_rows)
    # one order alone gives the same bytes
    assert np.array_equal(raw(mx.quantize(x, block_rows=block_rows).codes), raw(q.codes))
    alone = mx.quantize(x, block_rows=block_rows, order="cols")
    assert np.array_equal(raw(alone.codes), raw(qt.codes)) and torch.equal(alone.scales, qt.scales)


def test_ties_go_to_even(mx):
    """Quotients that lie half-way between two codes, exactly: multiples of half a step below a largest value of 448."""
    y = np.concatenate([(8 + np.arange(8) + 0.5) * 2.0 ** e for e in range(-9, 5)])
    y = np.concatenate([y, (np.arange(8) + 0.5) * 2.0 ** -9])
    y = y[y < 448]
    for top in (448.0, 1.0, 3.0, 1.5 * 2.0 ** 20, 127.0 * 2.0 ** -40):
        x = np.zeros((1, 128))
        x[0, 0] = top
        x[0, 1:1 + len(y)] = y * top / 448.0
        exact = x.astype(np.float32).astype(np.float64) == x  # products that fp32 holds
        q = mx.quantize(torch.from_numpy(x.astype(np.float32)).cuda())
        got = O.TABLE[raw(q.codes)][0]
        unit = np.append(np.append(448.0, y), np.zeros(127 - len(y)))
        low = np.floor(unit / O.step(unit)) * O.step(unit)
        even = np.where(np.floor(unit / O.step(unit)) % 2 == 0, low, low + O.step(unit))
        want = np.where(unit / O.step(unit) % 1 == 0.5, even, unit)
        assert np.array_equal(got[exact[0]], want[exact[0]]) and exact[0].sum() > 8


@pytest.mark.parametrize("order", ["rows", "both"])
def test_strided_unaligned_and_listed_sources(mx, order):
    big = matrix(70, 517, BF16, 3)
    x = big[3:68, 5:390]  # rows of odd stride that start off 16 bytes
    got = mx.quantize(x, order=order)
    want = mx.quantize(x.clone(), order=order)
    for a, b in zip(got if order == "both" else (got,), want if order == "both" else (want,)):
        assert np.array_equal(raw(a.codes), raw(b.codes)) and torch.equal(a.scales, b.scales)
    ms = [matrix(65, 200, F32, s) for s in range(3)]
    many = mx.quantize(ms, block_rows=128, order=order)
    batch = mx.quantize(torch.stack(ms), block_rows=128, order=order)
    for a, b in zip(many if order == "both" else (many,), batch if order == "both" else (batch,)):
        assert a.codes.shape[0] == 3 and np.array_equal(raw(a.codes), raw(b.codes)) and torch.equal(a.scales, b.scales)
    one = mx.quantize(ms[1], block_rows=128)
    first = many[0] if order == "both" else many
    assert np.array_equal(raw(first[1].codes), raw(one.codes)) and torch.equal(first[1].scales, one.scales)


@pytest.mark.parametrize("order", ["rows", "cols", "both"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gathered_rows(mx, order, weighted, dtype):
    g = torch.Generator().manual_seed(5)
    x = matrix(37, 200, dtype, 9)
    pairs = torch.randint(-2, 37 * 3, (150,), generator=g).to(torch.int32)
    pairs[7] = 37 * 3 + 5  # behind x
    w = torch.randn(37, 3, generator=g)
    ref = O.gather(x.double().cpu().numpy(), pairs.numpy(), 3, w.double().numpy() if weighted else None)
    # the product with the weight is rounded to fp32 before the block's maximum is taken
    ref = ref.astype(np.float32).astype(np.float64)
    if weighted:
        got = mx.quantize(x, order=order, pairs=pairs.cuda(), weights=w.cuda())
    else:
        got = mx.quantize(x, order=order, pairs=(pairs.cuda(), 3))
    got = got if order == "both" else (got,)
    if order != "cols":
        check_codes(got[0], ref, 1)
    if order != "rows":
        check_codes(got[-1], ref.T, 1)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_extreme_blocks(mx, block_rows):
    """Blocks of zeros, below the smallest scale, up to the largest float, and with NaN or an infinity in them."""
    x = torch.zeros(6 * 128, 128)
    x[128:256] = 2.0 ** -101
    x[256:384] = torch.randn(128, 128) * 2.0 ** -99
    x[384:512] = 3.4e38
    x[512:640] = torch.randn(128, 128)
    x[640:] = torch.randn(128, 128)
    x[512 + 5, 7] = math.nan
    x[640 + 5, 9] = -math.inf
    for order in ("rows", "both"):
        q = mx.quantize(x.cuda(), block_rows=block_rows, order=order)
        q = q if order == "both" else (q,)
        v = q[0].float().cpu()
        assert not v[:256].any()
        err = (v[256:512].double() - x[256:512].double()).abs()
        assert (err <= x[256:512].double().abs() * 2.0 ** -4 * (1 + 2.0 ** -20) +
                q[0].scales.cpu().double().t().repeat_interleave(block_rows, 0)[256:512] * 2.0 ** -10).all()
        bad = torch.zeros(768, dtype=torch.bool)
        if block_rows == 1:
            bad[517] = bad[645] = True
        else:
            bad[512:] = True
        assert v[bad].isnan().all() and v[~bad].isfinite().all()
        if order == "both":
            t = q[1].float().cpu().t()
            assert torch.equal(t.isnan(), bad[:, None].expand(-1, 128) if block_rows == 128 else
                               torch.cat([torch.zeros(512, 128), torch.ones(128, 1) * (torch.arange(128) == 7),
                                          torch.ones(128, 1) * (torch.arange(128) == 9)]).bool())


# ------------------------------------------------------------ products

def coded(mx, rows, cols, block_rows, seed, count=None):
    x = torch.stack([matrix(rows, cols, F32, seed + i) for i in range(count or 1)])
    return mx.quantize(x if count else x[0], block_rows=block_rows)


def of(q, i=None):
    codes, scales = (q.codes, q.scales) if i is None else (q.codes[i], q.scales[i])
    return O.values(raw(codes), scales.cpu().numpy(), q.block_rows)


def check_product(c, want, size, lost, cols, before=None):
    """Off by the roundings of the additions and of the products with the scales, an ulp (2^-23) of the sum of
    magnitudes each, and by half an ulp of the result's type; a bf16 result also by what the instruction for 8-bit
    floats drops (oracle/blocks.py)."""
    blocks = -(-cols // 128)
    tol = (lost if c.dtype == BF16 else 0) + size * (128 + blocks + 4) * 2.0 ** -23
    want = want if before is None else want + before
    tol = tol + np.abs(want) * torch.finfo(c.dtype).eps / 2 + (0 if before is None else np.abs(before) * 2.0 ** -23)
    err = np.abs(c.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err - tol).max())


PRODUCTS = [(1, 1, 1), (1, 4096, 512), (5, 17, 129), (16, 128, 256), (33, 100, 1000), (64, 300, 640), (65, 257, 384),
            (128, 128, 128), (130, 1000, 100), (257, 511, 2049), (700, 900, 300)]


@pytest.mark.parametrize("out", [BF16, F32, "add"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(mx, m, n, k, block_rows, out):
    a, b = coded(mx, m, k, 1, m + n), coded(mx, n, k, block_rows, k)
    want, size, lost = O.product(of(a), of(b))
    if out == "add":
        base = torch.randn(m, n + 3, generator=torch.Generator().manual_seed(1)).cuda()[:, 1:n + 1]
        c = base.clone()
        got = mx.block_matmul(a, b, out=c, accumulate=True)
        assert got is c
        check_product(c, want, size, lost, k, base.double().cpu().numpy())
    else:
        check_product(mx.block_matmul(a, b, dtype=out), want, size, lost, k)


@pytest.mark.parametrize("m,n,k,block_rows", [(4000, 4096, 256, 128), (4000, 4100, 640, 1)])
def test_large_tiles(mx, m, n, k, block_rows):
    a, b = coded(mx, m, k, 1, 2), coded(mx, n, k, block_rows, 3)
    va, vb = of(a), of(b)
    for dtype in (BF16, F32):
        c = mx.block_matmul(a, b, dtype=dtype)
        for rows in (slice(0, 40), slice(250, 290), slice(m - 300, m)):  # first tile, a border, the last tiles
            check_product(c[rows], *O.product(va[rows], vb), k)


def test_result_stays_inside_its_rows(mx):
    a, b = coded(mx, 130, 200, 1, 2), coded(mx, 77, 200, 128, 3)
    for dtype in (BF16, F32):
        whole = torch.full((133, 90), 7.0, dtype=dtype, device="cuda")
        mx.block_matmul(a, b, out=whole[2:132, 5:82])
        left = whole.clone()
        left[2:132, 5:82] = 7.0
        assert (left == 7.0).all()
        assert torch.equal(whole[2:132, 5:82], mx.block_matmul(a, b, dtype=dtype))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_batches(mx, block_rows):
    a, b = coded(mx, 70, 300, 1, 2, count=3), coded(mx, 150, 300, block_rows, 9, count=3)
    c = mx.block_matmul(a, b, dtype=F32)
    for i in range(3):
        check_product(c[i], *O.product(of(a, i), of(b, i)), 300)
        assert torch.equal(c[i], mx.block_matmul(a[i], b[i], dtype=F32))


def segments(lengths, align, tail):
    at = [0]
    for n in lengths:
        at.append(at[-1] + -(-n // align) * align)
    return at, at[-1] + tail


EXPERTS = [([5], 1, 0), ([1, 0, 0, 3, 2], 1, 3), ([0, 0, 0], 1, 4), ([300, 1, 0, 129, 256, 40], 1, 7),
           ([1] * 70 + [0] * 60, 1, 0), ([1000, 700], 1, 1)]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("n,k", [(96, 200), (300, 129)])
@pytest.mark.parametrize("lengths,align,tail", EXPERTS)
def test_expert_rows(mx, lengths, align, tail, n, k, block_rows):
    at, rows = segments(lengths, align, tail)
    a, b = coded(mx, rows, k, 1, 1), coded(mx, n, k, block_rows, 50, count=len(lengths))
    offsets = torch.tensor(at, dtype=torch.int32).cuda()
    for dtype in (BF16, F32):
        c = torch.full((rows, n), 3.0, dtype=dtype, device="cuda")
        mx.expert_matmul(a, b, offsets, out=c)
        assert (c[at[-1]:] == 3.0).all()  # behind the last expert
        va = of(a)
        for e in range(len(lengths)):
            if at[e + 1] > at[e]:
                check_product(c[at[e]:at[e + 1]], *O.product(va[at[e]:at[e + 1]], of(b, e)), k)


@pytest.mark.parametrize("lengths", [[5], [0, 130, 0, 1, 700, 0], [0, 0], [1] * 40])
@pytest.mark.parametrize("m,n", [(96, 200), (300, 129)])
def test_expert_gradients(mx, lengths, m, n):
    at, rows = segments(lengths, 128, 128)
    x = matrix(rows, m, F32, 1)
    y = matrix(rows, n, F32, 2)
    a, b = mx.quantize(x, order="cols"), mx.quantize(y, order="cols")
    va, vb = of(a), of(b)
    offsets = torch.tensor(at, dtype=torch.int32).cuda()
    base = torch.randn(len(lengths), m, n, generator=torch.Generator().manual_seed(1)).cuda()
    added = base.clone()
    mx.expert_grad(a, b, offsets, out=added, accumulate=True)
    fresh = mx.expert_grad(a, b, offsets)
    low = mx.expert_grad(a, b, offsets, dtype=BF16)
    for e in range(len(lengths)):
        lo, hi = at[e], at[e + 1]
        if hi == lo:
            assert torch.equal(added[e], base[e]) and not fresh[e].any() and not low[e].any()
            continue
        want, size, lost = O.product(va[:, lo:hi], vb[:, lo:hi])
        check_product(fresh[e], want, size, lost, hi - lo)
        check_product(low[e], want, size, lost, hi - lo)
        check_product(added[e], want, size, lost, hi - lo, base[e].double().cpu().numpy())


def test_offsets_outside_are_taken_as_the_nearest_bound(mx):
    a, b = coded(mx, 50, 256, 1, 1), coded(mx, 40, 256, 128, 2, count=3)
    wild = torch.tensor([-5, 20, 10, 1 << 30], dtype=torch.int32).cuda()
    c = torch.zeros(50, 40, dtype=F32, device="cuda")
    mx.expert_matmul(a, b, wild, out=c)  # 0..20, none, 10..50
    want = torch.zeros_like(c)
    mx.expert_matmul(a, b, torch.tensor([0, 10, 10, 50], dtype=torch.int32).cuda(), out=want)
    assert torch.equal(c[20:], want[20:])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_not_finite_reach_the_result(mx, bad):
    x = matrix(200, 384, F32, 1)
    x[17, 200] = bad
    w = matrix(100, 384, F32, 2)
    c = mx.block_matmul(mx.quantize(x), mx.quantize(w, block_rows=128))
    assert c[17].isnan().all() and c[:17].isfinite().all() and c[18:].isfinite().all()
    w[50, 130] = bad
    c = mx.block_matmul(mx.quantize(matrix(200, 384, F32, 1)), mx.quantize(w, block_rows=128))
    assert c.isnan().all()


def test_empty_sizes(mx):
    empty = torch.empty(0, 256, device="cuda")
    q, qt = mx.quantize(empty, order="both")
    assert q.codes.shape == (0, 256) and qt.codes.shape == (256, 0)
    b = coded(mx, 40, 256, 128, 2)
    assert mx.block_matmul(q, b).shape == (0, 40)
    b3 = coded(mx, 40, 256, 128, 2, count=2)
    assert mx.expert_matmul(q, b3, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 40)
    out = torch.ones(2, 256, 256, device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert (mx.expert_grad(qt, qt, o, out=out, accumulate=True) == 1).all()
    assert not mx.expert_grad(qt, qt, o, out=out).any()


def test_captured_and_on_another_stream(mx):
    x, w = matrix(200, 500, BF16, 1), matrix(300, 500, BF16, 2)
    qx, qw = mx.BlockCodes.empty(200, 500), mx.BlockCodes.empty(300, 500, 128)
    c = torch.empty(200, 300, dtype=BF16, device="cuda")

    def run(stream=None):
        mx.quantize(x, out=qx, stream=stream)
        mx.quantize(w, block_rows=128, out=qw, stream=stream)
        mx.block_matmul(qx, qw, out=c, stream=stream)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in (5, 6, 7):
        x.copy_(matrix(200, 500, BF16, seed))
        w.copy_(matrix(300, 500, BF16, seed + 10))
        g.replay()
        got = c.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        c.zero_()
        side.wait_stream(torch.cuda.current_stream())
        run(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, c)
        want = mx.block_matmul(mx.quantize(x), mx.quantize(w, block_rows=128))
        assert torch.equal(got, want)


def test_bits_repeat(mx):
    a, b = coded(mx, 300, 2000, 1, 1), coded(mx, 500, 2000, 128, 2)
    first = mx.block_matmul(a, b, dtype=F32)
    assert all(torch.equal(first, mx.block_matmul(a, b, dtype=F32)) for _ in range(5))
