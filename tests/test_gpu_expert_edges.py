"""GPU tests of the expert operators at the edges of their contracts: tokens
that went nowhere with logits that are no numbers, results and memory on
another stream than the current one, no tokens, no columns, segments that do
not start on whole blocks, quotients half-way between two codes."""

import math

import numpy as np
import pytest
import torch

from oracle import blocks as O
from oracle import experts as X
from tests.test_gpu_blocks import check_product, coded, matrix, of, raw

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


# ------------------------------------------------------------ the router's gradient

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,experts,k", [(6, 40, 4), (90, 300, 8)])
def test_gradient_of_masked_rows_that_are_not_numbers(mx, tokens, experts, k, dtype, renormalize, score):
    """Padding holds anything: its weights are 0, so its logits' gradient is, whatever they are."""
    z = torch.randn(tokens, experts, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    z[1] = math.nan
    z[2, 3] = math.inf
    z[3, 5] = math.nan
    z[4] = math.inf
    mask = torch.ones(tokens, dtype=torch.bool)
    mask[1:5] = False
    g = torch.randn(tokens, k, generator=torch.Generator().manual_seed(2))
    r = mx.route(z, k, score=score, renormalize=renormalize, scale=1.5, mask=mask.cuda())
    assert (r.experts[1:5] == -1).all() and not r.weights[1:5].any()
    got = mx.route_backward(z, r, g.cuda())
    assert not got[1:5].any()
    z[1:5] = 0.0  # the other rows are what they are without such padding
    assert torch.equal(got, mx.route_backward(z, mx.route(z, k, score=score, renormalize=renormalize, scale=1.5,
                                                          mask=mask.cuda()), g.cuda()))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_rows_that_are_not_numbers_without_a_mask(mx, renormalize, score):
    z = torch.randn(6, 40, generator=torch.Generator().manual_seed(1)).cuda()
    z[1, 3] = math.nan
    z[2] = -math.inf
    r = mx.route(z, 4, score=score, renormalize=renormalize)
    got = mx.route_backward(z, r, torch.ones(6, 4).cuda())
    assert got[1].isnan().all() and not got[2].any() and got[[0, 3, 4, 5]].isfinite().all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,top,k", [(32, 5, 3), (64, 31, 16), (96, 2, 6), (160, 7, 8), (480, 32, 16)])
def test_as_many_groups_as_there_may_be(mx, experts, top, k, score):
    """32 groups of 1 to 15 experts: lanes behind the last expert belong to no group."""
    z = torch.randn(100, experts, generator=torch.Generator().manual_seed(experts)).cuda()
    bias = (0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(1))).cuda()
    for kw in (dict(), dict(bias=bias), dict(group_best=1)):
        r = mx.route(z, k, groups=32, top_groups=top, score=score, **kw)
        ref = dict(kw, bias=bias.double().cpu().numpy()) if "bias" in kw else kw
        want, _ = X.route(z.double().cpu().numpy(), k, groups=32, top_groups=top, score=score, **ref)
        assert np.array_equal(r.experts.cpu().numpy(), want)


# ------------------------------------------------------------ streams

def owner(t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no memory of the allocator")


@pytest.mark.parametrize("handle", [False, True])
def test_results_are_memory_of_the_calls_stream(mx, handle):
    """A block that the current stream's queued kernels still use must not go to a call on another stream."""
    s = torch.cuda.Stream()
    stream = s.cuda_stream if handle else s
    x, w = matrix(200, 256, BF16, 1), matrix(96, 256, BF16, 2)
    z = torch.randn(200, 8, device="cuda")
    b3 = mx.quantize(torch.stack([w, w, w, w, w, w, w, w]), block_rows=128)
    torch.cuda.synchronize()
    q, qt = mx.quantize(x, order="both", stream=stream)
    b = mx.quantize(w, block_rows=128, stream=stream)
    c = mx.block_matmul(q, b, stream=stream)
    r = mx.route(z, 2, align=128, stream=stream)
    a, at = mx.quantize(x, pairs=(r.pairs, 2), order="both", stream=stream)
    y = mx.expert_matmul(a, b3, r.offsets, stream=stream)
    dw = mx.expert_grad(at, at, r.offsets, stream=stream)
    out = mx.expert_sum(y, r.slots, r.weights, stream=stream)
    dots = mx.expert_dot(out, y, r.slots, stream=stream)
    dz = mx.route_backward(z, r, dots, stream=stream)
    none = mx.route(z[:0], 2, align=8, stream=stream)
    nothing = mx.expert_sum(y[:0], r.slots, stream=stream)
    zeros = mx.block_matmul(mx.BlockCodes.empty(5, 0), mx.BlockCodes.empty(7, 0), stream=stream)
    made = [q.codes, q.scales, qt.codes, qt.scales, b.codes, c, r.experts, r.weights, a.codes, at.scales, y, dw, out, dots,
            dz, none.pairs, nothing, zeros]
    assert {owner(t) for t in made} == {s.cuda_stream} and owner(x) == torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    assert torch.equal(c, mx.block_matmul(mx.quantize(x), mx.quantize(w, block_rows=128)))


def test_results_of_another_stream_outlive_their_use_on_the_current_one(mx):
    """Dropped while the current stream still reads it: its memory must not go to the other stream's next call."""
    x = matrix(512, 2048, BF16, 1)
    side = torch.cuda.Stream()
    want = mx.quantize(x).codes.view(torch.uint8).clone()
    torch.cuda.synchronize()
    q = mx.quantize(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    got = q.codes.view(torch.uint8).clone()
    del q
    with torch.cuda.stream(side):
        junk = [torch.full((512, 2048), 3, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 8


@pytest.mark.parametrize("explicit", [True, False])
def test_dropped_codes_and_biases_outlive_their_kernels(mx, explicit):
    """WeightCodes and BalanceBias, and the control block that a bias follows, are dropped while their kernels still wait
    on a side stream: their memory must not go to new tensors before these ran."""
    ws = [matrix(256, 512, BF16, s) for s in range(4)]
    codes, bias, control = mx.WeightCodes(ws), mx.BalanceBias(512, rate=0.5), mx.StepControl("cuda")
    sizes = [t.untyped_storage().nbytes() for t in (codes.codes.codes, codes.codes.scales, codes.batch.owned[0],
                                                    bias.bias, bias.loads, control.block)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        if not explicit:
            codes.refresh()
            bias.step(control)
    if explicit:
        codes.refresh(stream=side)
        bias.step(control, stream=side)
    del codes, bias, control
    junk = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(24)]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in junk)


def test_a_dropped_step_with_codes_on_a_side_stream(mx):
    w = [matrix(128, 256, F32, s) for s in range(3)]
    g = [0.01 * torch.randn_like(t) for t in w]
    bias = mx.BalanceBias(256, rate=0.5)
    opt = mx.OptimizerStep([(f"layers.{i}.w", a, b) for i, (a, b) in enumerate(zip(w, g))], max_grad_norm=1.0,
                           codes={"w": [f"layers.{i}.w" for i in range(3)]}, balance=[bias])
    sizes = [t.untyped_storage().nbytes() for t in (opt.codes["w"].codes.codes, opt.codes["w"].codes.scales,
                                                    opt.codes["w"].batch.owned[0], bias.bias, bias.loads)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        opt.step()
    del opt, bias
    junk = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(24)]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in junk)


# ------------------------------------------------------------ empty batches

@pytest.mark.parametrize("on_stream", [False, True])
@pytest.mark.parametrize("align", [1, 8, 128])
def test_a_layer_of_no_tokens(mx, align, on_stream):
    """An empty micro-batch goes through the whole layer, forward and backward, and adds nothing."""
    experts, k, width, outs = 5, 2, 200, 136
    side = torch.cuda.Stream() if on_stream else None
    w = mx.WeightCodes(torch.randn(experts, outs, width, device="cuda"))
    x, z = torch.empty(0, width, dtype=BF16, device="cuda"), torch.empty(0, experts, device="cuda")
    grad = torch.empty(0, outs, dtype=BF16, device="cuda")
    loads = torch.zeros(experts, dtype=I32, device="cuda")
    dw = torch.ones(experts, outs, width, device="cuda")
    junk = torch.full((1 << 22,), 0x55, dtype=torch.uint8, device="cuda")  # what new memory would hold
    torch.cuda.synchronize()
    del junk
    kw = dict(stream=side)
    r = mx.route(z, k, align=align, loads=loads, **kw)
    a, at = mx.quantize(x, pairs=(r.pairs, k), order="both", **kw)
    rows = -(-experts * (align - 1) // align) * align
    assert r.pairs.numel() == rows and (a.rows, a.cols, at.rows, at.cols) == (rows, width, width, rows)
    y = mx.expert_matmul(a, w.codes, r.offsets, **kw)
    out = mx.expert_sum(y, r.slots, r.weights, **kw)
    g, gt = mx.quantize(grad, pairs=r.pairs, weights=r.weights, order="both", **kw)
    mx.expert_grad(gt, at, r.offsets, out=dw, accumulate=True, **kw)
    fresh = mx.expert_grad(gt, at, r.offsets, **kw)
    dx = mx.expert_sum(mx.expert_matmul(g, w.transposed, r.offsets, **kw), r.slots, **kw)
    dz = mx.route_backward(z, r, mx.expert_dot(grad, y, r.slots, **kw), **kw)
    torch.cuda.synchronize()
    assert (out.shape, dx.shape, dz.shape) == ((0, outs), (0, width), (0, experts)) and not loads.any()
    assert (dw == 1).all() and not fresh.any()
    for q in (a, at, g, gt):  # rows of -1 are zeros, the padding too
        whole = q.codes.as_strided((q.rows, -(-q.cols // 128) * 128), q.codes.stride())
        assert not raw(whole).any() and not q.scales.any()


def test_zero_rows_for_pairs_into_given_codes(mx):
    x = torch.empty(0, 300, device="cuda")
    pairs = torch.full((7,), -1, dtype=I32, device="cuda")
    q, qt = mx.BlockCodes.empty(7, 300), mx.BlockCodes.empty(300, 7)
    wide = q.codes.as_strided((7, 384), (384, 1))
    for t in (wide.view(torch.uint8), qt.codes.as_strided((300, 128), (128, 1)).view(torch.uint8)):
        t.fill_(0x55)
    q.scales.fill_(5.0)
    qt.scales.fill_(5.0)
    mx.quantize(x, pairs=pairs, order="both", out=(q, qt))
    assert not raw(wide).any() and not q.scales.any() and not qt.scales.any()
    assert not raw(qt.codes.as_strided((300, 128), (128, 1))).any()
    # codes inside a wider buffer: what lies around them stays
    big = torch.full((9, 640), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((3, 10), 5.0, device="cuda")
    part = mx.BlockCodes(big[1:8, 128:428], scales[:, 2:9])
    mx.quantize(x, pairs=pairs, out=part)
    left = raw(big)
    assert not left[1:8, 128:512].any() and (left[[0, 8]] == 0x55).all()
    assert (left[:, :128] == 0x55).all() and (left[:, 512:] == 0x55).all()
    assert not scales[:, 2:9].any() and (scales[:, :2] == 5).all() and (scales[:, 9] == 5).all()


def test_products_of_no_columns(mx):
    a, b = mx.BlockCodes.empty(6, 0), mx.BlockCodes.empty(7, 0, 128, 3)
    o = torch.tensor([1, 3, 3, 5], dtype=I32).cuda()
    for dtype in (F32, BF16):
        assert not mx.expert_matmul(a, b, o, dtype=dtype)[1:5].any()
        out = torch.full((6, 7), 4.0, dtype=dtype, device="cuda")
        got = mx.expert_matmul(a, b, o, out=out)
        assert got is out and not out[1:5].any() and (out[[0, 5]] == 4).all()  # rows of no expert stay
    out = torch.full((6, 7), 4.0, device="cuda")
    assert (mx.expert_matmul(a, b, o, out=out, accumulate=True) == 4).all()


# ------------------------------------------------------------ gradients over segments anywhere

SEGMENTS = [([5], 0, 0), ([5, 0, 130, 0, 1, 70], 0, 0), ([100, 27, 1, 300], 3, 77), ([0, 0, 0], 130, 200), ([1] * 40, 0, 9),
            ([64, 64, 128, 129, 127, 0, 1], 1, 1), ([1, 600], 127, 0)]


@pytest.mark.parametrize("lengths,lead,tail", SEGMENTS)
@pytest.mark.parametrize("m,n", [(96, 200), (300, 129)])
def test_expert_gradients_of_any_segments(mx, m, n, lengths, lead, tail):
    """Segments that start and end inside a block of 128 rows (an order of align=1): each expert's rows alone count."""
    at = [lead]
    for length in lengths:
        at.append(at[-1] + length)
    rows = at[-1] + tail
    a, b = mx.quantize(matrix(rows, m, F32, 1), order="cols"), mx.quantize(matrix(rows, n, F32, 2), order="cols")
    va, vb = of(a), of(b)
    offsets = torch.tensor(at, dtype=I32).cuda()
    base = torch.randn(len(lengths), m, n, generator=torch.Generator().manual_seed(1)).cuda()
    added = base.clone()
    mx.expert_grad(a, b, offsets, out=added, accumulate=True)
    fresh, low = mx.expert_grad(a, b, offsets), mx.expert_grad(a, b, offsets, dtype=BF16)
    for e in range(len(lengths)):
        lo, hi = at[e], at[e + 1]
        if hi == lo:
            assert torch.equal(added[e], base[e]) and not fresh[e].any() and not low[e].any()
            continue
        # rounding: a segment meets at most one block more than its length fills
        want, size, lost = O.product(np.pad(va, ((0, 0), (0, 8)))[:, lo:hi], np.pad(vb, ((0, 0), (0, 8)))[:, lo:hi])
        # the instruction's eight products are those of the whole rows: of the segment's, or of zeros
        first, last = lo // 8 * 8, -(-hi // 8) * 8
        inside = (np.arange(first, last) >= lo) & (np.arange(first, last) < hi)
        lost = O.product((np.pad(va, ((0, 0), (0, 8)))[:, first:last] * inside),
                         (np.pad(vb, ((0, 0), (0, 8)))[:, first:last] * inside))[2]
        check_product(fresh[e], want, size, lost, hi - lo + 128)
        check_product(low[e], want, size, lost, hi - lo + 128)
        check_product(added[e], want, size, lost, hi - lo + 128, base[e].double().cpu().numpy())


def test_expert_gradients_of_an_order_without_alignment(mx):
    """route() as it is by default, and the gradient over its order."""
    tokens, experts, k, width, outs = 300, 7, 2, 130, 90
    x, grad = matrix(tokens, width, BF16, 3), matrix(tokens, outs, BF16, 4)
    r = mx.route(torch.randn(tokens, experts, generator=torch.Generator().manual_seed(5)).cuda(), k)
    _, xt = mx.quantize(x, pairs=(r.pairs, k), order="both")
    _, gt = mx.quantize(grad, pairs=r.pairs, weights=r.weights, order="both")
    got = mx.expert_grad(gt, xt, r.offsets)
    va, vb, at = of(gt), of(xt), r.offsets.tolist()
    for e in range(experts):
        lo, hi = at[e], at[e + 1]
        want, size, lost = O.product(va[:, lo:hi], vb[:, lo:hi])
        check_product(got[e], want, size, lost, hi - lo + 128)


# ------------------------------------------------------------ ties of codes

def ties():
    """Rows of 128 fp32 values with 24-bit significands: the first is the largest, 28 m, and 448 x / max|x| of each other
    one lies exactly half-way between two codes."""
    rng = np.random.default_rng(0)
    odd, rows = np.arange(17, 32, 2), []
    for r in range(256):
        m = float(rng.integers(1 << 18, (1 << 24) // 31) | 1)
        t = np.concatenate([odd * 2.0 ** (e - 1) for e in range(-6, 5)] + [(2 * np.arange(8) + 1) * 2.0 ** -10])
        t = rng.permutation(t[t < 448])[:127]
        t = np.concatenate([[448.0], t, np.zeros(127 - len(t))]) * rng.choice([-1.0, 1.0], 128)
        rows.append(t)
        rows[-1] = (t, m * 2.0 ** float(rng.integers(-90, 90)))
    unit = np.stack([t for t, _ in rows])
    factor = np.array([f for _, f in rows])[:, None]
    return unit, factor


def half_to_even(unit):
    whole = np.floor(np.abs(unit) / O.step(unit))
    even = np.where(np.abs(unit) / O.step(unit) % 1 == 0.5, whole + whole % 2, np.abs(unit) / O.step(unit))
    return np.copysign(even * O.step(unit), unit)


@pytest.mark.parametrize("order", ["rows", "cols", "both"])
def test_ties_of_long_significands_go_to_even(mx, order):
    unit, factor = ties()
    x = (unit * factor / 16).astype(np.float32)
    assert np.array_equal(x.astype(np.float64), unit * factor / 16)  # all of them floats, and 448 x / max is unit
    want = half_to_even(unit)
    if order != "cols":
        q = mx.quantize(torch.from_numpy(x).cuda(), order=order)
        q = q[0] if order == "both" else q
        assert np.array_equal(O.TABLE[raw(q.codes)], want)
    if order != "rows":  # the same blocks as columns
        q = mx.quantize(torch.from_numpy(x.T.copy()).cuda(), order=order)
        q = q[1] if order == "both" else q
        assert np.array_equal(O.TABLE[raw(q.codes)], want)
    if order == "rows":  # one block of 128 x 128
        same = np.concatenate([unit[:1], unit[1:128]])
        block = (same * factor[0] / 16).astype(np.float32)
        q = mx.quantize(torch.from_numpy(block).cuda(), block_rows=128)
        assert np.array_equal(O.TABLE[raw(q.codes)], half_to_even(same))


@pytest.mark.parametrize("order", ["rows", "both"])
def test_ties_of_weighted_bf16_rows_go_to_even(mx, order):
    unit, factor = ties()
    unit = np.where(np.abs(unit) >= 2.0 ** -6, unit, 0.0)
    pairs = torch.arange(256, dtype=I32).cuda()
    w = torch.from_numpy(factor.astype(np.float32)).cuda()
    x = torch.from_numpy(unit / 16).to(BF16)
    assert np.array_equal(x.double().numpy(), unit / 16)
    q = mx.quantize(x.cuda(), pairs=pairs, weights=w, order=order)
    assert np.array_equal(O.TABLE[raw((q[0] if order == "both" else q).codes)], half_to_even(unit))


# ------------------------------------------------------------ columns past 32 bits of bytes

def test_a_result_of_more_than_2_31_bytes_a_row_accumulates(mx):
    """Column offsets in bytes pass 32 bits: 66 GiB of codes, all but the last rows zeros."""
    n = (1 << 29) + 300
    a = mx.quantize(torch.ones(1, 128, device="cuda"))
    codes = torch.zeros(n, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    few = mx.quantize(torch.arange(1, 401, dtype=F32, device="cuda")[:, None].expand(400, 128).contiguous())
    codes[-400:] = few.codes
    scales = torch.zeros(1, n, device="cuda")
    scales[:, -400:] = few.scales
    out = torch.ones(1, n, device="cuda")
    mx.block_matmul(a, mx.BlockCodes(codes, scales), out=out, accumulate=True)
    want = 1 + 128.0 * torch.arange(1, 401, device="cuda")
    assert torch.all((out[0, -400:] - want).abs() <= 1e-5 * want)
    assert bool((out[0, :-400] == 1).all())
    del codes, scales, out
    torch.cuda.empty_cache()


# ------------------------------------------------------------ weighted rows

@pytest.mark.parametrize("order", ["rows", "both"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_rows_weight_falls_out_of_its_own_blocks_codes(mx, dtype, order):
    """code = round(448 w x / max|w x|): whatever the weight, a positive one gives the codes of the row alone, ties
    among them, and a negative one their opposites."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(200, 300, generator=g).to(dtype)
    x[3] = 0.0
    x[4, 128:256] = 2.0 ** -99  # a whole block near the smallest
    w = torch.randn(200, 1, generator=g) * torch.exp2(torch.randint(-20, 20, (200, 1), generator=g).float())
    pairs = torch.arange(200, dtype=I32)
    alone = mx.quantize(x.cuda())
    got = mx.quantize(x.cuda(), pairs=pairs.cuda(), weights=w.cuda(), order=order)
    got = got[0] if order == "both" else got
    want = O.TABLE[raw(alone.codes)] * np.sign(w.numpy())
    top = (x.abs().float() * w.abs()).numpy()  # products rounded to fp32, as the scale takes them
    scale = O.tops(top.astype(np.float64), 1)
    scale[scale < O.TINY] = 0.0
    want = np.where(O.spread(scale, want.shape, 1) == 0, 0.0, want)
    keep = np.ones(200, dtype=bool)
    keep[4] = False  # its block's codes are zeros or those of the rounded products
    assert np.array_equal(O.TABLE[raw(got.codes)][keep], want[keep])
    assert np.array_equal(got.scales.cpu().numpy(), scale.astype(np.float32) / np.float32(448.0))


@pytest.mark.parametrize("order", ["rows", "cols", "both"])
def test_weights_out_of_range(mx, order):
    """Weights of zero, not numbers, infinities, and such that take a row's values out of the range at either end."""
    x = torch.randn(12, 128, generator=torch.Generator().manual_seed(1))
    x[:, 5] = 0.0
    x[8:10] *= 2.0 ** -110  # below the smallest block by itself
    x[10] *= 2.0 ** 100
    w = torch.tensor([1.0, 0.0, math.nan, math.inf, -math.inf, 2.0 ** -120, -0.0, -2.0, 2.0 ** 60, 1.0, 2.0 ** 100, 2.0 ** -40])
    got = mx.quantize(x.cuda(), pairs=torch.arange(12, dtype=I32).cuda(), weights=w[:, None].cuda(), order=order)
    rows = None if order == "cols" else (got[0] if order == "both" else got)
    cols = None if order == "rows" else (got[1] if order == "both" else got)
    if rows is not None:
        v = rows.float().cpu()
        assert v[[2, 3, 4, 10]].isnan().all()                      # (2^100 times 2^100 is no float)
        assert not v[[1, 5, 6, 9]].any() and not rows.scales[0, [1, 5, 6, 9]].any()
        for r in (0, 7, 8, 11):
            true = x[r].double() * w[r].double()
            top = true.abs().max()
            assert (v[r].double() - true).abs().max() <= top * 2.0 ** -4 and v[r].isfinite().all()
            assert abs(rows.scales[0, r].item() - top.item() / 448.0) <= top.item() / 448.0 * 2.0 ** -22
    if cols is not None:  # a column's block holds all the rows
        v = cols.float().cpu()
        assert v.isnan().all()
