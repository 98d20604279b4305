"""GPU tests of the expert operators together, as a training step uses them: a
mixture-of-experts layer forward and backward in 8-bit block codes, its weight
gradients added to the buffers that a clipped optimizer step reads, the codes
made anew and the balance bias moved by that step; eager, captured, on another
stream."""

import numpy as np
import pytest
import torch

from oracle import blocks as B
from oracle import experts as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TOKENS, EXPERTS, K, WIDTH, OUT = 300, 12, 3, 200, 136


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


def raw(codes):
    return codes.contiguous().view(torch.uint8).cpu().numpy()


def of(q, i=None):
    codes, scales = (q.codes, q.scales) if i is None else (q.codes[i], q.scales[i])
    return B.values(raw(codes), scales.cpu().numpy(), q.block_rows)


class Layer:
    """out[t] = sum over the chosen experts of w[t, j] * W[e] x[t]; the router is a matrix too."""

    def __init__(self, mx, state_bits=32, **kw):
        self.mx = mx
        g = torch.Generator().manual_seed(0)
        self.weight = (0.1 * torch.randn(EXPERTS, OUT, WIDTH, generator=g)).cuda()
        self.router = (0.1 * torch.randn(EXPERTS, WIDTH, generator=g)).cuda()
        self.weight_grad = torch.zeros_like(self.weight)
        self.router_grad = torch.zeros_like(self.router)
        self.balance = mx.BalanceBias(EXPERTS, rate=0.01)
        params = [(f"experts.{e}.w", self.weight[e], self.weight_grad[e]) for e in range(EXPERTS)]
        params += [("router.w", self.router, self.router_grad)]
        self.opt = mx.OptimizerStep(params, max_grad_norm=1.0, skip_nonfinite=True, muon_lr=0.01,
                                    codes={"experts": [f"experts.{e}.w" for e in range(EXPERTS)], "router": "router.w"},
                                    balance=[self.balance], **kw)
        self.codes = self.opt.codes["experts"]

    def forward_backward(self, x, grad):
        mx = self.mx
        logits = x.float() @ self.router.t()
        r = mx.route(logits, K, score="sigmoid", bias=self.balance.bias, loads=self.balance.loads, align=128)
        a, at = mx.quantize(x, pairs=(r.pairs, K), order="both")
        y = mx.expert_matmul(a, self.codes.codes, r.offsets)
        out = mx.expert_sum(y, r.slots, r.weights)
        g, gt = mx.quantize(grad, pairs=r.pairs, weights=r.weights, order="both")
        mx.expert_grad(gt, at, r.offsets, out=self.weight_grad, accumulate=True)
        grad_rows = mx.expert_matmul(g, self.codes.transposed, r.offsets)
        grad_logits = mx.route_backward(logits, r, mx.expert_dot(grad, y, r.slots))
        grad_x = mx.expert_sum(grad_rows, r.slots, dtype=F32) + grad_logits @ self.router
        self.router_grad.add_(grad_logits.t() @ x.float())
        return dict(logits=logits, r=r, a=a, at=at, y=y, out=out, g=g, gt=gt, rows=grad_rows, grad_logits=grad_logits,
                    grad_x=grad_x)

    def step(self, x, grad):
        self.weight_grad.zero_()
        self.router_grad.zero_()
        for part in range(2):  # two micro-batches
            self.forward_backward(x[part], grad[part])
        self.opt.step()


def batch(seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(2, TOKENS, WIDTH, generator=g).to(BF16).cuda(),
            (0.01 * torch.randn(2, TOKENS, OUT, generator=g)).to(BF16).cuda())


def near(got, want, tol):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) - tol).max())


def test_layer_and_its_gradients(mx):
    layer = Layer(mx)
    xs, grads = batch(1)
    x, grad = xs[0], grads[0]
    got = layer.forward_backward(x, grad)
    r = got["r"]
    xd, gd = x.double().cpu().numpy(), grad.double().cpu().numpy()
    chosen, w = O.route(got["logits"].double().cpu().numpy(), K, score="sigmoid", bias=np.zeros(EXPERTS))
    assert np.array_equal(r.experts.cpu().numpy(), chosen)
    slots, pairs, offsets, loads = O.order(chosen, EXPERTS, 128)
    assert np.array_equal(r.pairs.cpu().numpy(), pairs) and np.array_equal(layer.balance.loads.cpu().numpy(), loads)
    wd = r.weights.double().cpu().numpy()
    near(wd, w, 1e-5)

    # the codes are the gathered rows' to half a step, in both orders
    for q, source, factors in ((got["a"], xd, None), (got["g"], gd, wd)):
        rows = B.gather(source, pairs, K, factors)
        unit = B.spread(q.scales.double().cpu().numpy(), rows.shape, 1)
        assert np.all(np.abs(of(q) - rows) <= unit * 0.5 * B.step(rows / np.where(unit > 0, unit, 1)) * (1 + 1e-6) +
                      np.abs(rows) * 2.0 ** -22)
    # everything after that against fp64 on the same codes: a sum of K terms, each half an ulp of bf16, or rounded
    # in fp32 (the bounds of the products are in test_gpu_blocks.py; here 1e-3 of the sums of magnitudes covers them)
    a, at, g, gt = of(got["a"]), of(got["at"]), of(got["g"]), of(got["gt"])
    y = np.zeros((len(pairs), OUT))
    rows = np.zeros((len(pairs), WIDTH))
    size_y, size_r = np.zeros_like(y), np.zeros_like(rows)
    for e in range(EXPERTS):
        lo, hi = offsets[e], offsets[e + 1]
        we, wt = of(layer.codes.codes, e), of(layer.codes.transposed, e)
        assert np.allclose(we, wt.T, rtol=0, atol=0)  # one scale for a square block: both orders have the same values
        y[lo:hi], size_y[lo:hi] = a[lo:hi] @ we.T, np.abs(a[lo:hi]) @ np.abs(we).T
        rows[lo:hi], size_r[lo:hi] = g[lo:hi] @ wt.T, np.abs(g[lo:hi]) @ np.abs(wt).T
        dw, size = gt[:, lo:hi] @ at[:, lo:hi].T, np.abs(gt[:, lo:hi]) @ np.abs(at[:, lo:hi]).T
        near(layer.weight_grad[e], dw, size * 1e-4)
    used = offsets[EXPERTS]
    near(got["y"][:used], y[:used], np.abs(y[:used]) * 2.0 ** -8 + size_y[:used] * 1e-3)
    yd = got["y"].double().cpu().numpy()
    out, size = O.expert_sum(yd, slots, wd)
    near(got["out"], out, np.abs(out) * 2.0 ** -8 + size * 1e-6)
    dots, size = O.expert_dot(gd, yd, slots)
    dz = O.route_backward(got["logits"].double().cpu().numpy(), chosen, dots, "sigmoid", True, 1.0)
    near(got["grad_logits"], dz, np.abs(dots).max() * 1e-5)
    rd = got["rows"].double().cpu().numpy()
    gx, size = O.expert_sum(rd, slots)
    gx = gx + dz @ layer.router.double().cpu().numpy()
    near(got["grad_x"], gx, size * 1e-6 + np.abs(dots).max() * 1e-4)


def test_gradients_equal_differences(mx):
    """Of the loss <out, grad> by the logits (through the weights alone) and by an expert's matrix, on codes that
    hold their values exactly: small integers over powers of two."""
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-4, 5, (64, 128), generator=g).to(BF16).cuda()
    x[:, 0] = 448.0                                            # every row's scale is 1
    w = torch.randint(-3, 4, (4, 128, 128), generator=g).float()
    w[:, 0, 0] = 448.0
    w[:, :, 0] *= (torch.arange(128) == 0)
    w = w.cuda()
    grad = torch.randint(-2, 3, (64, 128), generator=g).to(BF16).cuda()
    z = torch.randn(64, 4, generator=g, dtype=torch.float64)
    codes = mx.WeightCodes(w)
    assert torch.equal(codes.codes.float(), w)

    def forward(z):
        r = mx.route(z.float().cuda(), 2, align=128)
        a = mx.quantize(x, pairs=(r.pairs, 2))
        return r, mx.expert_matmul(a, codes.codes, r.offsets, dtype=F32)

    r, y = forward(z)
    got = mx.route_backward(z.float().cuda(), r, mx.expert_dot(grad.float(), y, r.slots)).double().cpu()
    yd, gd = y.double().cpu().numpy(), grad.double().cpu().numpy()
    chosen, slots = r.experts.cpu().numpy(), r.slots.cpu().numpy()

    def loss(z):
        return (O.expert_sum(yd, slots, O.weights_of(z, chosen, "softmax", True, 1.0))[0] * gd).sum(1)

    h = 1e-5
    for e in range(4):
        up, down = z.numpy().copy(), z.numpy().copy()
        up[:, e] += h
        down[:, e] -= h
        d = (loss(up) - loss(down)) / (2 * h)
        scale = np.abs(yd).max() * 2 * 128
        assert np.abs(d - got[:, e].numpy()).max() <= scale * 1e-6
    # the weight gradient of sum_t w_t <grad_t, W x_t>: exact where the weights are powers of two
    weights = torch.full((64, 2), 0.5, device="cuda")
    _, at = mx.quantize(x, pairs=(r.pairs, 2), order="both")
    _, gt = mx.quantize(grad, pairs=r.pairs, weights=weights, order="both")
    dw = mx.expert_grad(gt, at, r.offsets)
    want = np.zeros((4, 128, 128))
    for t in range(64):
        for j in range(2):
            want[chosen[t, j]] += 0.5 * np.outer(gd[t], x[t].double().cpu().numpy())
    unit = np.abs(want).max()
    assert np.abs(dw.double().cpu().numpy() - want).max() <= unit * 2.0 ** -4  # e4m3's half step on each factor at most


def test_step_writes_codes_and_moves_the_bias(mx):
    layer = Layer(mx)
    before = layer.weight.clone()
    xs, grads = batch(2)
    layer.step(xs, grads)
    assert not torch.equal(layer.weight, before)
    fresh, turned = mx.quantize([layer.weight[e] for e in range(EXPERTS)], block_rows=128, order="both")
    for own, want in ((layer.codes.codes, fresh), (layer.codes.transposed, turned)):
        assert np.array_equal(raw(own.codes), raw(want.codes)) and torch.equal(own.scales, want.scales)
    assert np.array_equal(raw(layer.opt.codes["router"].codes.codes), raw(mx.quantize(layer.router, block_rows=128).codes))
    assert layer.balance.bias.abs().max() == np.float32(0.01) and not layer.balance.loads.any()
    norm = torch.sqrt(layer.weight_grad.double().square().sum() + layer.router_grad.double().square().sum())
    assert abs(layer.opt.clip.control.norm.item() - norm.item()) <= 1e-6 * norm.item()
    # a gradient that is not finite: weights, codes and bias stay
    kept = [t.clone() for t in (layer.weight, layer.router, layer.balance.bias)]
    codes = raw(layer.codes.codes.codes)
    xs[1, 5, 7] = float("nan")
    layer.step(xs, grads)
    assert layer.opt.clip.control.skip.item() == 1
    for own, want in zip((layer.weight, layer.router, layer.balance.bias), kept):
        assert torch.equal(own, want)
    assert np.array_equal(raw(layer.codes.codes.codes), codes)


def test_captured_steps_equal_eager_ones(mx):
    eager, captured = Layer(mx), Layer(mx)
    xs, grads = batch(3)
    x, grad = xs.clone(), grads.clone()
    captured.step(x, grad)  # warm up, then start again from the other's state
    torch.cuda.synchronize()
    captured.opt.load_state_dict(eager.opt.state_dict())
    captured.weight.copy_(eager.weight)
    captured.router.copy_(eager.router)
    for c in captured.opt.codes.values():
        c.refresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step(x, grad)
    for seed in (11, 12, 13):
        xs, grads = batch(seed)
        x.copy_(xs)
        grad.copy_(grads)
        graph.replay()
        torch.cuda.synchronize()
        eager.step(xs, grads)
        for name in ("weight", "router", "weight_grad", "router_grad"):
            assert torch.equal(getattr(captured, name), getattr(eager, name)), (seed, name)
        assert torch.equal(captured.balance.bias, eager.balance.bias)
        assert np.array_equal(raw(captured.codes.transposed.codes), raw(eager.codes.transposed.codes))


def test_another_stream_and_two_at_once(mx):
    xs, grads = batch(4)
    a, b = Layer(mx), Layer(mx)
    want = a.forward_backward(xs[0], grads[0])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    results = []
    for s, layer in ((s1, a), (s2, b)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            results.append(layer.forward_backward(xs[0], grads[0]))
    torch.cuda.synchronize()
    for got in results:
        for key in ("out", "grad_x", "grad_logits"):
            assert torch.equal(got[key], want[key])
    # the raw stream of a call's own argument, results recorded on it
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = mx.route(want["logits"], K, score="sigmoid", bias=a.balance.bias, align=128, stream=side)
    q = mx.quantize(xs[0], pairs=(r.pairs, K), stream=side)
    y = mx.expert_matmul(q, a.codes.codes, r.offsets, stream=side)
    out = mx.expert_sum(y, r.slots, r.weights, stream=side)
    del q, y
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want["out"])


def test_decoding_one_token(mx):
    layer = Layer(mx)
    x = batch(5)[0][0]
    many = layer.forward_backward(x, torch.zeros(TOKENS, OUT, dtype=BF16, device="cuda"))
    for t in (0, 17):
        r = mx.route(many["logits"][t:t + 1], K, score="sigmoid", bias=layer.balance.bias)
        a = mx.quantize(x[t:t + 1], pairs=(r.pairs, K))
        y = mx.expert_matmul(a, layer.codes.codes, r.offsets)
        out = mx.expert_sum(y, r.slots, r.weights)
        assert torch.equal(r.experts, many["r"].experts[t:t + 1]) and r.offsets[-1] == K
        # another kernel adds the blocks in another order: both are within half an ulp of bf16 of each row's value
        size = many["out"][t].double().abs() + many["y"][many["r"].slots[t].long()].double().abs().sum(0)
        assert ((out[0].double() - many["out"][t].double()).abs() <= size * 2.0 ** -7).all()
