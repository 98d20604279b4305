"""GPU parity of the routing to experts, its gradient, the order by expert, the
balance bias and the tokens' sums with plain fp64 implementations
(oracle/experts.py): ties, near ties, masks, groups, odd sizes, graphs."""

import math

import numpy as np
import pytest
import torch

from oracle import experts as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


def check_weights(got, want):
    """A score is off by the exponential's 1 ulp and the argument's rounding (|z| 2^-24, |z| <= 32 here), the sum by as
    much and an ulp for each of its up to 5 + 4 levels' additions, the quotient and the factor by half an ulp each:
    less than 2 * (2 + 32) + 9 + 2 half ulps together."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.all(np.abs(got[ok] - want[ok]) <= np.abs(want[ok]) * 80 * 2.0 ** -24 + 1e-37)


def check(mx, z, k, align=1, mask=None, loads=True, **kw):
    """route() against the oracle; returns its Routing."""
    experts = z.shape[1]
    counted = torch.full((experts,), 5, dtype=torch.int32, device="cuda") if loads else None
    bias = kw.get("bias")
    r = mx.route(z, k, align=align, mask=None if mask is None else mask.cuda(), loads=counted, **kw)
    ref = dict(kw)
    if bias is not None:
        ref["bias"] = bias.double().cpu().numpy()
    chosen, weights = O.route(z.double().cpu().numpy(), k, mask=None if mask is None else mask.numpy(), **ref)
    assert np.array_equal(r.experts.cpu().numpy(), chosen)
    check_weights(r.weights, weights)
    slots, pairs, offsets, load = O.order(chosen, experts, align)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.pairs.cpu().numpy(), pairs)
    if loads:
        assert np.array_equal(counted.cpu().numpy(), load + 5)
    return r


def logits(tokens, experts, dtype=F32, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(tokens, experts, generator=g)).to(dtype).cuda()


SIZES = [(1, 1, 1), (1, 64, 6), (3, 5, 5), (63, 17, 3), (64, 64, 16), (65, 65, 1), (130, 100, 8), (256, 128, 8),
         (257, 129, 9), (520, 256, 8), (300, 300, 12), (1000, 511, 4), (70, 512, 16)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k", SIZES)
def test_routes(mx, tokens, experts, k, score, dtype):
    z = logits(tokens, experts, dtype, tokens + experts)
    check(mx, z, k, score=score)
    check(mx, z, k, score=score, renormalize=False, scale=2.5, align=128)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k", SIZES)
def test_bias_chooses(mx, tokens, experts, k, score, dtype):
    z = logits(tokens, experts, dtype, tokens)
    bias = (0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(1))).cuda()
    check(mx, z, k, score=score, bias=bias)
    check(mx, z, k, score=score, bias=torch.zeros_like(bias), renormalize=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_best", [1, 2])
@pytest.mark.parametrize("experts,groups,top,k", [(256, 8, 4, 8), (160, 8, 3, 6), (33, 11, 2, 5), (512, 32, 5, 16),
                                                  (24, 24, 3, 3), (90, 3, 1, 9), (6, 2, 2, 4)])
def test_groups(mx, experts, groups, top, k, group_best, score, dtype):
    z = logits(150, experts, dtype, experts)
    kw = dict(groups=groups, top_groups=top, group_best=group_best, score=score)
    check(mx, z, k, **kw)
    bias = (0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(1))).cuda()
    check(mx, z, k, bias=bias, **kw)


@pytest.mark.parametrize("tokens", [5, 64, 65, 300])
def test_masked_tokens_and_experts(mx, tokens):
    z = logits(tokens, 40, F32, 3)
    z[:, 7] = -math.inf
    z[1] = -math.inf                     # nothing is left
    z[2, 3:] = -math.inf                 # three are left, five are asked for
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(2)) > 0.3
    mask[1:4] = True
    bias = (0.1 * torch.randn(40, generator=torch.Generator().manual_seed(1))).cuda()
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(bias=bias), dict(bias=bias, groups=4, top_groups=2), dict(groups=5, top_groups=1)):
            for align in (1, 128):
                check(mx, z, 5, mask=mask, score=score, align=align, **kw)
    none = torch.zeros(tokens, dtype=torch.bool)
    r = check(mx, z, 5, mask=none, align=128)
    assert (r.pairs == -1).all() and not r.offsets.any()


def test_all_tokens_to_one_expert(mx):
    z = torch.full((700, 30), -4.0)
    z[:, 11] = 9.0
    check(mx, z.cuda(), 1, align=128)
    check(mx, z.cuda(), 2)  # the second by a tie of all the others: expert 0


def test_ties(mx):
    z = torch.zeros(100, 64)
    check(mx, z.cuda(), 5)
    check(mx, z.cuda(), 5, bias=torch.zeros(64).cuda())
    check(mx, z.cuda(), 5, groups=8, top_groups=2)
    z = torch.randint(0, 3, (300, 100), generator=torch.Generator().manual_seed(1)).float()
    for kw in (dict(), dict(bias=torch.zeros(100).cuda()), dict(groups=10, top_groups=4)):
        for score in ("softmax", "sigmoid"):
            check(mx, z.cuda(), 7, score=score, **kw)


def test_keys_closer_than_fp32(mx):
    """Scores that fp32 cannot tell apart are told apart: expert e's bias makes up for its score but for 1e-10 * e."""
    z = logits(200, 32, F32, 5, 1.0)
    z[1:] = z[0] + 1e-7 * torch.arange(1, 200, device="cuda")[:, None]
    s = O.scores(z[:1].double().cpu().numpy(), "sigmoid")[0]
    bias = torch.from_numpy((0.5 - s).astype(np.float32)).cuda()
    check(mx, z, 8, score="sigmoid", bias=bias)
    check(mx, z, 8, score="sigmoid", bias=bias, groups=4, top_groups=2)
    check(mx, z, 8, score="softmax", bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_not_a_number(mx, score):
    z = logits(70, 40, F32, 1)
    z[3, 5] = math.nan
    z[4, 6] = math.inf
    z[66, 0] = -math.nan
    check(mx, z, 4, score=score)
    check(mx, z, 4, score=score, bias=torch.zeros(40).cuda(), groups=4, top_groups=2)
    bias = torch.zeros(40)
    bias[9] = math.nan
    check(mx, z[:5].contiguous(), 4, score=score, bias=bias.cuda())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k", [(40, 400, 16), (300, 200, 8), (300, 512, 8)])
def test_tokens_of_many_experts(mx, tokens, experts, k, score):
    """Masks, infinities, NaN, ties and near keys where a token is more than 16 lanes (tokens beyond 64 and a bias for
    200 experts, any call for 400)."""
    z = logits(tokens, experts, F32, 9)
    z[:, 7] = -math.inf
    z[1] = -math.inf
    z[2, 3:] = -math.inf
    z[3, 150] = math.nan
    z[4, experts - 1] = math.inf
    z[5] = 0.25
    z[6] = torch.randint(0, 3, (experts,), generator=torch.Generator().manual_seed(1)).float().cuda()
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(2)) > 0.3
    mask[1:7] = True
    bias = (0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(1))).cuda()
    for kw in (dict(), dict(bias=bias), dict(bias=torch.zeros_like(bias)), dict(bias=bias, groups=4, top_groups=2),
               dict(groups=8, top_groups=4), dict(groups=8, top_groups=1, group_best=1, bias=bias)):
        check(mx, z, k, mask=mask, score=score, align=128, **kw)
    z = logits(tokens, experts, F32, 5, 1.0)
    z[1:] = z[0] + 1e-7 * torch.arange(1, tokens, device="cuda")[:, None]
    s = O.scores(z[:1].double().cpu().numpy(), score)[0]
    bias = torch.from_numpy((0.5 - s).astype(np.float32)).cuda()
    check(mx, z, k, score=score, bias=bias)
    check(mx, z, k, score=score, bias=bias, groups=4, top_groups=2)


def test_results_without_a_kernel_on_a_stream(mx):
    """No tokens, no rows, no columns: the results are filled on the call's stream, not on the current one, which is
    busy here until long after."""
    z = torch.zeros(0, 6, device="cuda")
    y, slots = torch.zeros(0, 9, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    grad = torch.zeros(4, 9, device="cuda")
    a, b = mx.BlockCodes.empty(5, 0), mx.BlockCodes.empty(7, 0)
    kept = torch.full((64, 512), 7.0, device="cuda")  # freed below: new results take memory that is not zero
    torch.cuda.synchronize()
    del kept
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        torch.cuda._sleep(20_000_000)
        r = mx.route(z, 2, align=8, stream=stream)
        out = mx.expert_sum(y, slots, stream=stream)
        dots = mx.expert_dot(grad, y, slots, stream=stream)
        c = mx.block_matmul(a, b, stream=stream)
        with torch.cuda.stream(s):
            assert (r.pairs.cpu() == -1).all() and r.pairs.numel() == 48 and not r.offsets.cpu().any()
            assert not out.cpu().any() and not dots.cpu().any() and not c.cpu().any() and c.shape == (5, 7)
        torch.cuda.synchronize()


@pytest.mark.parametrize("experts", [3, 64])
def test_order_of_a_million_tokens(mx, experts):
    """More counts than the order's 16-bit counters take in one pass, from skewed tokens; the chosen are those of a
    stable sort."""
    tokens, k, align = (1 << 20) + 77, 2, 128
    z = torch.randn(tokens, experts, generator=torch.Generator().manual_seed(4)) - 0.05 * torch.arange(experts)
    r = mx.route(z.cuda(), k, align=align)
    chosen = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]  # (topk leaves the order of equals open)
    assert torch.equal(r.experts.cpu().long(), chosen)
    flat = chosen.flatten().numpy()
    counts = np.bincount(flat, minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    order = np.argsort(flat, kind="stable")
    first = np.concatenate([[0], np.cumsum(counts)])[:-1]
    slots = np.empty(tokens * k, np.int64)
    slots[order] = offsets[flat[order]] + np.arange(tokens * k) - first[flat[order]]
    assert np.array_equal(r.slots.cpu().numpy().ravel(), slots)
    pairs = np.full(r.pairs.numel(), -1, np.int64)
    pairs[slots] = np.arange(tokens * k)
    assert np.array_equal(r.pairs.cpu().numpy(), pairs)


def test_strided_logits_and_without_order(mx):
    big = logits(90, 101, BF16, 1)
    z = big[3:80, 7:90]
    assert z.data_ptr() % 16
    check(mx, z, 6)
    check(mx, z, 6, bias=torch.full((83,), 0.01).cuda())
    loads = torch.zeros(83, dtype=torch.int32, device="cuda")
    full, bare = mx.route(z, 6), mx.route(z, 6, order=False, loads=loads)
    assert bare.slots is None and bare.pairs is None and bare.offsets is None
    assert torch.equal(full.experts, bare.experts) and torch.equal(full.weights, bare.weights)
    assert torch.equal(loads, torch.bincount(full.experts.view(-1), minlength=83).int())
    g = torch.randn(77, 6).cuda()
    assert torch.equal(mx.route_backward(z, full, g), mx.route_backward(z.contiguous(), full, g))
    out = torch.full((77, 100), 7.0, dtype=BF16, device="cuda")
    mx.route_backward(z, full, g, out=out[:, 3:86])
    assert torch.equal(out[:, 3:86], mx.route_backward(z, full, g)) and (out[:, :3] == 7).all() and (out[:, 86:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (17, 5, 3), (100, 64, 6), (33, 129, 8), (70, 256, 16), (40, 500, 9)])
def test_gradient(mx, tokens, experts, k, renormalize, score, dtype):
    z = logits(tokens, experts, dtype, experts)
    if tokens > 3 and experts > k:
        z[1, :2] = -math.inf
        z[2] = -math.inf
    mask = torch.ones(tokens, dtype=torch.bool)
    mask[tokens // 2] = tokens == 1
    r = mx.route(z, k, score=score, renormalize=renormalize, scale=1.7, mask=mask.cuda())
    g = torch.randn(tokens, k, generator=torch.Generator().manual_seed(3))
    got = mx.route_backward(z, r, g.cuda())
    assert got.dtype == dtype
    zz = z.double().cpu().numpy()
    want = O.route_backward(zz, r.experts.cpu().numpy(), g.double().numpy(), score, renormalize, 1.7)
    # the weights' roundings (check_weights), times the gradients that are subtracted from each other
    size = np.abs(g.numpy()).max(1, keepdims=True) * 1.7 * 2
    tol = size * 100 * 2.0 ** -24 + np.abs(want) * torch.finfo(dtype).eps / 2
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def test_gradient_of_a_token_that_is_not_a_number(mx):
    z = logits(5, 40, F32, 1)
    z[3, 5] = math.nan
    r = mx.route(z, 4)
    got = mx.route_backward(z, r, torch.ones(5, 4).cuda())
    assert got[3].isnan().all() and got[[0, 1, 2, 4]].isfinite().all()


def test_no_tokens(mx):
    z = torch.empty(0, 40, device="cuda")
    r = mx.route(z, 4, align=128)
    assert r.experts.shape == (0, 4) and (r.pairs == -1).all() and r.offsets.shape == (41,) and not r.offsets.any()
    assert mx.route_backward(z, r, torch.empty(0, 4, device="cuda")).shape == (0, 40)
    assert mx.expert_sum(torch.empty(0, 8, device="cuda"), torch.full((3, 2), -1, dtype=torch.int32).cuda()).eq(0).all()


def test_loads_add_up_and_balance(mx):
    b = mx.BalanceBias(40, rate=0.01)
    total = np.zeros(40)
    for seed in range(3):
        z = logits(300, 40, F32, seed)
        r = mx.route(z, 4, score="sigmoid", bias=b.bias, loads=b.loads)
        total += np.bincount(r.experts.cpu().numpy().ravel(), minlength=40)
    assert np.array_equal(b.loads.cpu().numpy(), total)
    b.step()
    assert np.array_equal(b.bias.cpu().numpy(), O.balance(np.zeros(40), total, 0.01).astype(np.float32))
    assert not b.loads.any()
    # under a control block that skips the bias stays, the loads start again
    control = mx.StepControl("cuda")
    before = b.bias.clone()
    b.loads.copy_(torch.arange(40))
    control.skip.fill_(1)
    b.step(control)
    assert torch.equal(b.bias, before) and not b.loads.any()
    control.skip.fill_(0)
    b.loads.copy_(torch.arange(40))
    b.step(control)
    assert (b.bias[:20] > before[:20]).all() and (b.bias[20:] < before[20:]).all()
    # equal loads move nothing, also where their mean is no integer
    b.loads.fill_(7)
    before = b.bias.clone()
    b.step()
    assert torch.equal(b.bias, before)


@pytest.mark.parametrize("y_type", [F32, BF16])
@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 1), (5, 3, 7), (33, 8, 512), (64, 16, 513), (130, 6, 2048), (9, 2, 5001)])
def test_sums_and_dots(mx, tokens, k, cols, out_type, y_type):
    g = torch.Generator().manual_seed(tokens + cols)
    rows = tokens * k + 3
    y = torch.randn(rows + 1, cols + 3, generator=g).to(y_type).cuda()[1:, 1:cols + 1]
    slots = torch.randint(-1, rows + 2, (tokens, k), generator=g).to(torch.int32)  # also behind y, and rows twice
    w = torch.randn(tokens, k, generator=g)
    yy = y.double().cpu().numpy()
    for weights in (w, None):
        want, size = O.expert_sum(yy, slots.numpy(), None if weights is None else weights.double().numpy())
        out = torch.full((tokens + 1, cols + 2), 7.0, dtype=out_type, device="cuda")
        mx.expert_sum(y, slots.cuda(), None if weights is None else weights.cuda(), out=out[1:, 1:cols + 1])
        tol = size * k * 2.0 ** -23 + np.abs(want) * torch.finfo(out_type).eps / 2
        assert np.all(np.abs(out[1:, 1:cols + 1].double().cpu().numpy() - want) <= tol)
        assert (out[0] == 7).all() and (out[:, 0] == 7).all() and (out[:, -1] == 7).all()
    grad = torch.randn(tokens, cols, generator=g).to(out_type).cuda()
    want, size = O.expert_dot(grad.double().cpu().numpy(), yy, slots.numpy())
    got = mx.expert_dot(grad, y, slots.cuda())
    depth = cols // 64 + 8 + 6  # additions in a row in a lane, and across the lanes
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= size * (depth + 1) * 2.0 ** -23)


def test_sum_passes_on_a_nan_weight(mx):
    y = torch.ones(4, 16, device="cuda")
    slots = torch.tensor([[0, 1], [-1, -1], [2, -1]], dtype=torch.int32).cuda()
    w = torch.tensor([[1.0, 2.0], [math.nan, math.nan], [3.0, 0.0]]).cuda()
    out = mx.expert_sum(y, slots, w)
    assert (out[0] == 3).all() and out[1].isnan().all() and (out[2] == 3).all()
    y[3] = math.nan  # a row that no slot names
    assert (mx.expert_sum(y, slots, w)[0] == 3).all()


def test_captured_routing(mx):
    z = logits(300, 64, BF16, 0)
    b = mx.BalanceBias(64, rate=0.01)
    control = mx.StepControl("cuda")

    def run():
        r = mx.route(z, 4, score="sigmoid", bias=b.bias, loads=b.loads, align=128)
        b.step(control)
        return r

    run()
    torch.cuda.synchronize()
    b.bias.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = run()
    bias = np.zeros(64)
    for seed in (5, 6, 7, 8):
        z.copy_(logits(300, 64, BF16, seed))
        g.replay()
        chosen, _ = O.route(z.double().cpu().numpy(), 4, score="sigmoid", bias=bias)
        assert np.array_equal(r.experts.cpu().numpy(), chosen)
        slots, pairs, offsets, loads = O.order(chosen, 64, 128)
        assert np.array_equal(r.slots.cpu().numpy(), slots) and np.array_equal(r.pairs.cpu().numpy(), pairs)
        bias = (bias.astype(np.float32) + np.float32(0.01) * np.sign(loads.mean() - loads).astype(np.float32))
        assert np.array_equal(b.bias.cpu().numpy(), bias)
        bias = bias.astype(np.float64)
