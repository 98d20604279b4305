"""GPU tests of the gradient norm (muon_grad_norm) and the many-tensor AdamW
(muon_adamw_multi) against the fp64 oracles.

Tolerances, all derived from roundings of relative size at most u = 2^-24
(fp32) or 2^-8 (bf16's half step, 2^-9 of the binade's top):

* m: beta1*m and (1-beta1)*g each carry at most 5 roundings (decoding, the
  constant, scale*g, the product, the sum), so |err| <= 5u (|beta1 m| +
  |(1-beta1) g|); 8u is asked.
* v has positive terms: at most 8 roundings relative to v (r^2 doubles the
  decoding's), and below the normal range each is 2^-150 at most; r = sqrt(v)
  carries v's error and two roundings of its own.
* theta: the step l*c1*m / (r*sqrt(c2) + eps) carries m's and r's errors and at
  most 12 further roundings of the step, (1-l*wd)*theta at most 3 roundings, and the
  result one of theta's type.
* a scale: the block's largest magnitude (its error as above) / 448: 3u more.
* a code: floor(|y|/q + u20) is monotone in |y|, so with |y| off by at most d
  the code lies between the codes of |y| - d and |y| + d for the same bits.
"""

import math

import numpy as np
import pytest
import torch

from oracle import adamw_multi as OM

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy().reshape(-1)


def codes(t):
    return t.view(torch.uint8).cpu().numpy().reshape(-1)


def half_step(x, dtype):
    """Half a step of dtype at |x|."""
    x = np.abs(x)
    e = np.floor(np.log2(np.where(x > 0, x, 1.0)))
    if dtype == F32:
        return np.maximum(np.where(x > 0, 2.0 ** (e - 24), 0.0), 2.0 ** -150)
    return np.maximum(np.where(x > 0, 2.0 ** (e - 8), 0.0), 2.0 ** -134)


def snapshot(opt, i):
    st = [x.clone() for x in opt._state(i)]
    return opt.params[i].detach().clone(), opt.grads[i].detach().clone(), st


def check_step(opt, i, before, t, scale=1.0, lr=None):
    """Tensor i of opt after one step from the state `before`, element by element."""
    p0, g0, st = before
    lr = (opt.lr if lr is None else lr) * opt.lr_factors[i]
    (b1, b2), eps, wd = opt.betas, opt.eps, opt.weight_decays[i]
    p, g, n = f64(p0), f64(g0) * scale, p0.numel()
    if n == 0:
        return
    if opt.bits[i] == 32:
        m, v = f64(st[0]), f64(st[1])
    else:
        s = st[2].to(torch.float64).cpu().numpy()
        m = OM.code_value(codes(st[0])) * OM.per_block(s[:, 0], n)
        v = (OM.code_value(codes(st[1])) * OM.per_block(s[:, 1], n)) ** 2
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    r1 = np.sqrt(v1)
    dm = 8 * U * (np.abs(b1 * m) + np.abs((1 - b1) * g)) + 2.0 ** -149
    dv = 8 * U * v1 + 2.0 ** -147  # up to four roundings below fp32's normal range
    dr = np.sqrt(v1 + dv) - np.sqrt(np.maximum(v1 - dv, 0.0)) + 2 * U * r1
    c1, c2 = 1 / (1 - b1 ** t), 1 / (1 - b2 ** t)
    den = r1 * math.sqrt(c2) + eps
    upd = lr * c1 * m1 / den
    want = (1 - lr * wd) * p - upd
    dp = abs(lr) * c1 * dm / den + np.abs(upd) * (12 * U + dr * math.sqrt(c2) / den) + 3 * U * np.abs(p) + 2.0 ** -149
    dp = dp + half_step(np.abs(want) + dp, p0.dtype)
    got = f64(opt.params[i])
    assert np.all(np.abs(got - want) <= dp), (i, np.max(np.abs(got - want) / dp))
    now = opt._state(i)
    if opt.bits[i] == 32:
        assert np.all(np.abs(f64(now[0]) - m1) <= dm)
        assert np.all(np.abs(f64(now[1]) - v1) <= dv)
        return
    scales = now[2].to(torch.float64).cpu().numpy()
    bits = OM.random_bits(opt._at[i] + np.arange(n), t, opt.seed)
    for k, (x, dx, least) in enumerate(((m1, dm, 0.0), (r1, dr, OM.LEAST))):
        pad = np.zeros(-(-n // 256) * 256)
        pad[:n] = np.abs(x)
        top = pad.reshape(-1, 256).max(1)
        pad[:n] = dx
        dtop = pad.reshape(-1, 256).max(1)
        sure = (top > OM.TINY * 1.01) | (top < OM.TINY * 0.99)  # on the border either is right
        want_s = np.where(top < OM.TINY, 0.0, top / OM.TOP)
        assert np.all(np.abs(scales[:, k] - want_s)[sure] <= (dtop / OM.TOP + 3 * U * want_s)[sure])
        s = scales[:, k]
        y = np.abs(x) / np.where(OM.per_block(s, n) == 0, np.inf, OM.per_block(s, n))
        dy = np.where(y == 0, 0.0, dx / np.where(OM.per_block(s, n) == 0, np.inf, OM.per_block(s, n)) + 4 * U * y)

        def code(a):
            return np.where(a <= 0, 0.0, OM.round_code(np.clip(a, least, OM.TOP), bits[k]))
        value = OM.code_value(codes(now[k]))
        live = OM.per_block(s, n) > 0
        lo, hi = code(np.maximum(y - dy, 0.0)), code(y + dy)
        if least:
            lo = np.where(y > 0, np.maximum(lo, least), 0.0)
        assert np.all((np.abs(value) >= lo)[live] & (np.abs(value) <= hi)[live]), (i, k)
        assert np.all(value[~live] == 0.0)
        sign = np.sign(value) * np.sign(x)
        assert np.all((sign >= 0)[np.abs(x) > dx])


SIZES = [(1,), (2,), (7,), (15,), (16,), (17,), (255,), (256,), (257,), (0,), (4095,), (4096,), (4097,), (3, 5), (64, 129),
         (12345,), (2, 4096)]


def make(dtypes, sizes, seed, offset=0):
    """Parameters and gradients of alternating types; with offset, views that
    start `offset` elements into a larger buffer (their memory is not 16-byte aligned)."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, s in enumerate(sizes):
        pair = []
        for dt, scale in zip(dtypes[i % len(dtypes)], (0.5, 10.0 ** (i % 5 - 3))):
            n = int(np.prod(s))
            buf = torch.full((n + offset + 3,), 77.0, dtype=dt, device="cuda")
            view = buf[offset:offset + n].view(s)
            view.copy_((scale * torch.randn(s, generator=gen)).to(dt))
            pair.append((view, buf))
        out.append(pair)
    return [a for (a, _), _ in out], [b for _, (b, _) in out], [x for pair in out for _, x in pair]


MIXED = [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)]


def refill(grads, seed):
    gen = torch.Generator().manual_seed(seed)
    for i, g in enumerate(grads):
        g.copy_((10.0 ** (i % 5 - 3) * torch.randn(g.shape, generator=gen)).to(g.dtype))


@pytest.mark.parametrize("bits", [32, 8, "both"])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_three_steps_of_mixed_types(mx, bits, offset):
    print(f"adamw_multi bits {bits} offset {offset}", flush=True)
    params, grads, buffers = make(MIXED, SIZES, 5, offset)
    n = len(params)
    widths = [8 if i % 3 else 32 for i in range(n)] if bits == "both" else bits
    opt = mx.AdamWMulti(params, grads, lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=[0.1 * (i % 2) for i in range(n)],
                        lr_factor=[1.0 + 0.5 * (i % 3) for i in range(n)], state_bits=widths, seed=12)
    for t in (1, 2, 3):
        refill(grads, 40 + t)
        before = [snapshot(opt, i) for i in range(n)]
        opt.step()
        torch.cuda.synchronize()
        for i in range(n):
            check_step(opt, i, before[i], t)
    for i, b in enumerate(buffers):  # memory around the tensors is as it was
        k = SIZES[i // 2]
        used = int(np.prod(k))
        assert torch.all(b[:offset] == 77.0) and torch.all(b[offset + used:] == 77.0)
    for buf, fill in ((opt.exp_avg, 0), (opt.codes_m, 0), (opt.codes_r, 0)):  # so are the gaps of the state
        if buf is None:
            continue
        mine = torch.ones(buf.numel(), dtype=torch.bool)
        for i in range(n):
            if (opt.bits[i] == 32) == (buf is opt.exp_avg):
                mine[opt._at[i]:opt._at[i] + params[i].numel()] = False
        assert torch.all(buf.view(torch.uint8 if buf.element_size() == 1 else F32).cpu()[mine] == fill)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas,eps,wd", [((0.0, 0.0), 1e-8, 0.0), ((0.95, 0.9999), 1e-15, 0.3), ((0.9, 0.95), 1e-2, 0.0)])
def test_hyperparameters_and_late_steps(mx, bits, betas, eps, wd):
    params, grads, _ = make(MIXED, [(5000,), (300,)], 9)
    opt = mx.AdamWMulti(params, grads, lr=3e-3, betas=betas, eps=eps, weight_decay=wd, state_bits=bits, seed=2 ** 32 - 1)
    for t in (1, 2, 100000):
        opt.t = t - 1
        before = [snapshot(opt, i) for i in range(2)]
        opt.step()
        torch.cuda.synchronize()
        for i in range(2):
            check_step(opt, i, before[i], t)


def test_zero_gradients_sparse_rows_and_tiny_values(mx):
    n = 256 * 12 + 100
    g = torch.zeros(n, device="cuda")
    g[256:512] = 1e-20           # squares below fp32's smallest normal
    g[512:768] = 1e-33           # the block is below 2^-100: it holds zeros
    g[768:1024] = 1e18           # large
    g[1024] = 3.0                # one element of its block
    g[2048:] = torch.randn(n - 2048, device="cuda")
    p = torch.randn(n, device="cuda")
    opt = mx.AdamWMulti([p], [g], lr=1e-2, weight_decay=0.1, state_bits=8, eps=1e-8)
    for t in (1, 2, 3):
        before = [snapshot(opt, 0)]
        opt.step()
        torch.cuda.synchronize()
        check_step(opt, 0, before[0], t)
        if t == 2:
            g.zero_()
    assert torch.all(opt.codes_m.view(torch.uint8)[:256] == 0) and torch.all(opt.scales[0] == 0)
    assert torch.all(opt.scales[2] == 0)
    assert torch.isfinite(p).all()


def test_nonfinite_gradients_stay_in_their_block(mx):
    n = 256 * 5
    for bad in (math.nan, math.inf, -math.inf):
        g = torch.randn(n, device="cuda")
        p = torch.randn(n, device="cuda")
        g[300] = bad
        opt = mx.AdamWMulti([p], [g], state_bits=8)
        opt.step()
        g[300] = 0.0
        opt.step()
        torch.cuda.synchronize()
        ok = torch.ones(n, dtype=torch.bool, device="cuda")
        ok[256:512] = False
        assert torch.isfinite(p[ok]).all()
        assert not torch.isfinite(p[300]) and not torch.isfinite(opt.scales[1]).any()
        m, v = opt.moments(0)
        assert torch.isfinite(m[ok]).all() and torch.isfinite(v[ok]).all()
        assert not torch.isfinite(m[256:512]).any()


def test_codes_are_unbiased(mx):
    """One block's values rounded with 4096 seeds: each mean within 6 standard
    errors of the value (an error of a code is below one step q, so its
    standard deviation is at most q/2), and the bits are the oracle's."""
    seeds = 4096
    g = torch.linspace(0.001, 1.0, 256, device="cuda")
    total = torch.zeros(2, 256, dtype=torch.float64, device="cuda")
    opt = mx.AdamWMulti([torch.zeros(256, device="cuda")], [g], lr=0.0, betas=(0.0, 0.0), state_bits=8)
    for s in range(seeds):
        opt.hyper.seed = s
        opt.t = 0
        opt.step()
        total[0] += opt.codes_m.double() * opt.scales[0, 0]
        total[1] += opt.codes_r.double() * opt.scales[0, 1]
    want = f64(g)
    s = float(opt.scales[0, 0])
    q = 2.0 ** (np.maximum(np.floor(np.log2(want / s)), -6) - 3) * s
    for k in range(2):
        assert np.all(np.abs(f64(total[k]) / seeds - want) <= 6 * q / 2 / math.sqrt(seeds) + 8 * U * want)


def test_moments_are_those_of_elementwise_tensor_code(mx):
    """m, v, the codes and the scales bit for bit as separate tensor operations
    give them (each product and sum rounded by itself), over several steps."""
    n, b1, b2 = 256 * 40, 0.9, 0.999
    gen = torch.Generator("cuda").manual_seed(5)
    wide, narrow = (mx.AdamWMulti([torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")], betas=(b1, b2),
                                  state_bits=bits, seed=77) for bits in (32, 8))
    m = torch.zeros(n, device="cuda")
    v = torch.zeros_like(m)
    dm, dr = torch.zeros_like(m), torch.zeros_like(m)  # what the codes stand for
    for t in range(1, 6):
        g = torch.randn(n, generator=gen, device="cuda") * torch.exp(torch.randn(n, generator=gen, device="cuda"))
        for opt in (wide, narrow):
            opt.grads[0].copy_(g)
            opt.step()
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        assert torch.equal(wide.exp_avg, m) and torch.equal(wide.exp_avg_sq, v)
        m8, r8 = dm * b1 + g * (1 - b1), (dr.square() * b2 + g * g * (1 - b2)).sqrt()
        decoded = []
        for x, bits, least, got, k in zip((m8, r8), OM.random_bits(np.arange(n), t, 77), (0.0, OM.LEAST),
                                          (narrow.codes_m, narrow.codes_r), (0, 1)):
            top = x.view(-1, 256).abs().amax(1, keepdim=True)
            s = top / 448.0
            y = (x.view(-1, 256) * (448.0 / top)).view(-1).cpu().numpy()
            a = np.where(y == 0, 0.0, np.clip(np.abs(y.astype(np.float64)), least, OM.TOP))
            want = torch.from_numpy(np.copysign(OM.round_code(a, bits), y)).to(torch.float32).cuda()
            assert torch.equal(got.float(), want)
            assert torch.equal(narrow.scales[:, k], s.view(-1))
            decoded.append((want.view(-1, 256) * s).view(-1))
        dm, dr = decoded


def test_more_than_2_to_31_elements(mx):
    """One tensor longer than 32-bit offsets reach: its last blocks against the
    oracle, and the positions of the random bits with them."""
    n = 2 ** 31 + 4096 + 77
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    tail = 3 * 256 + 77
    g[-tail:] = torch.randn(tail, device="cuda").to(BF16)
    g[:256] = 1.0
    opt = mx.AdamWMulti([p], [g], lr=1e-2, state_bits=8, seed=4)
    clip = mx.GradClip([g], max_norm=0.5)
    clip.step()
    opt.step()
    torch.cuda.synchronize()
    want = OM.grad_norm([f64(g[-tail:]), f64(g[:256])], 0.5)
    assert abs(float(clip.control.norm) - want[0]) <= 2 * U * want[0]
    z = np.zeros(tail, dtype=np.uint8)
    ref = OM.adamw8_step(np.zeros(tail), f64(g[-tail:]), z, z, np.zeros((4, 2)), 1, 1e-2, 0.9, 0.999, 1e-8, 0.0,
                         counter=n - tail, seed=4)
    got = OM.code_value(codes(opt.codes_m[n - tail:n]))
    assert np.mean(got != ref["codes_m"]) <= 0.01  # a rounding on the border may go either way; other bits would differ in a third
    assert np.all(np.abs(f64(p[-tail:]) - ref["param"]) <= 2.0 ** -8 * np.abs(ref["param"]))
    assert torch.all(p[256:4096] == 0) and torch.all(opt.codes_r.view(torch.uint8)[256:4096] == 0)
    assert torch.all(p[:256] != 0)


# ------------------------------------------------------------ norm and control

@pytest.mark.parametrize("offset", [0, 1])
def test_grad_norm_of_mixed_types(mx, offset):
    _, grads, _ = make(MIXED, SIZES + [(3, 16384), (100001,)], 3, offset)
    for max_norm in (0.25, 1e9, math.inf):
        clip = mx.GradClip(grads, max_norm=max_norm)
        clip.step()
        torch.cuda.synchronize()
        norm, scale = OM.grad_norm([f64(g) for g in grads], max_norm)
        c = clip.control
        # fp64 sums, one rounding to fp32, and one of the quotient
        assert abs(float(c.norm) - norm) <= U * norm
        assert abs(float(c.scale) - scale) <= 3 * U * scale
        assert (int(c.step), int(c.skip), int(c.skipped)) == (1, 0, 0)


def test_grad_norm_limits(mx):
    """Values whose squares leave fp32's range, and more chunks than workgroups."""
    for value in (3e38, 1e-30):
        g = torch.full((3000,), value, device="cuda")
        clip = mx.GradClip([g[:0], g, g[:0]], max_norm=1.0)
        clip.step()
        norm = float(g[0].double()) * math.sqrt(3000)
        if norm < 3.4e38:
            assert abs(float(clip.control.norm) - norm) <= 2 * U * norm
            assert float(clip.control.scale) == 1.0
        else:
            assert float(clip.control.norm) == math.inf
    g = torch.full((1,), 3e38, device="cuda")
    clip = mx.GradClip([g])
    clip.step()
    assert float(clip.control.norm) == float(g[0])
    empty = mx.GradClip([g[:0]], max_norm=1.0)
    empty.step()
    assert float(empty.control.norm) == 0.0 and float(empty.control.scale) == 1.0 and int(empty.control.step) == 1
    big = torch.randn(16384 * 2500 + 5, device="cuda")
    small = [torch.randn(3, device="cuda") for _ in range(2100)]
    clip = mx.GradClip([big, *small], max_norm=1.0)
    clip.step()
    want = math.sqrt(float(big.double().square().sum()) + sum(float(s.double().square().sum()) for s in small))
    assert abs(float(clip.control.norm) - want) <= 2 * U * want


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nonfinite_norms(mx, bad):
    g = [torch.randn(5000, device="cuda"), torch.randn(70, device="cuda").to(BF16)]
    g[1][69] = bad
    clip = mx.GradClip(g, max_norm=1.0, skip_nonfinite=True)
    clip.step()
    c = clip.control
    assert (int(c.step), int(c.skip), int(c.skipped)) == (0, 1, 1)
    assert math.isnan(float(c.norm)) if math.isnan(bad) else float(c.norm) == math.inf
    g[1][69] = 0.0
    clip.step()
    assert (int(c.step), int(c.skip), int(c.skipped)) == (1, 0, 1) and math.isfinite(float(c.norm))
    plain = mx.GradClip(g, max_norm=1.0)
    g[1][69] = bad
    plain.step()
    assert (int(plain.control.step), int(plain.control.skip)) == (1, 0)
    if math.isnan(bad):
        assert math.isnan(float(plain.control.scale))
    else:
        assert float(plain.control.scale) == 0.0


@pytest.mark.parametrize("bits", [32, 8])
def test_control_scale_step_factor_and_skip(mx, bits):
    params, grads, _ = make(MIXED, SIZES, 8)
    control = mx.StepControl("cuda", step=41)
    clip = mx.GradClip(grads, max_norm=0.5, skip_nonfinite=True, control=control)
    opt = mx.AdamWMulti(params, grads, lr=1e-2, weight_decay=0.1, state_bits=bits, seed=3, control=control)
    control.lr_factor.fill_(0.25)
    before = [snapshot(opt, i) for i in range(len(params))]
    clip.step()
    opt.step()
    torch.cuda.synchronize()
    assert int(control.step) == 42
    for i in range(len(params)):
        check_step(opt, i, before[i], 42, scale=float(control.scale), lr=1e-2 * 0.25)
    # a gradient that is not finite: nothing changes, the step is not counted
    before = [snapshot(opt, i) for i in range(len(params))]
    grads[7][3] = math.nan
    clip.step()
    opt.step()
    torch.cuda.synchronize()
    assert (int(control.step), int(control.skipped), int(control.skip)) == (42, 1, 1)
    for i, (p0, _, st) in enumerate(before):
        assert torch.equal(params[i], p0)
        for x, y in zip(st, opt._state(i)):
            assert torch.equal(x.view(torch.uint8), y.contiguous().view(torch.uint8))
    # and the next good one counts on
    grads[7][3] = 0.5
    clip.step()
    opt.step()
    torch.cuda.synchronize()
    assert int(control.step) == 43 and not torch.equal(params[7], before[7][0])


def test_equal_inputs_give_equal_bits_on_any_stream(mx):
    def run(side):
        params, grads, _ = make(MIXED, SIZES + [(70000,)], 8)
        clip = mx.GradClip(grads, max_norm=0.5)
        opt = mx.AdamWMulti(params, grads, state_bits=[8 if i % 2 else 32 for i in range(len(params))], control=clip.control)
        torch.cuda.synchronize()
        for t in range(3):
            clip.step(stream=side)
            opt.step(stream=side)
        torch.cuda.synchronize()
        return params, opt, clip

    a, b = run(None), run(torch.cuda.Stream())
    for x, y in zip(a[0], b[0]):
        assert torch.equal(x, y)
    assert torch.equal(a[1].codes_m.view(torch.uint8), b[1].codes_m.view(torch.uint8))
    assert torch.equal(a[1].exp_avg, b[1].exp_avg) and torch.equal(a[2].control.norm, b[2].control.norm)


@pytest.mark.parametrize("explicit", [True, False])
def test_dropped_objects_outlive_their_kernels(mx, explicit):
    """The optimizer is dropped while its step still waits on a side stream:
    its state's memory must not go to the next allocation before the step ran."""
    n = 1 << 20
    p, twin, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda"), torch.randn(n, device="cuda")
    one = mx.AdamWMulti([twin], [g], lr=1e-2)
    one.step()
    opt = mx.AdamWMulti([p], [g], lr=1e-2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        if not explicit:
            opt.step()
    if explicit:
        opt.step(stream=side)
    del opt
    junk = [torch.full((n,), 1e30, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(p, twin) and len(junk) == 8


def test_two_steps_at_once_on_two_streams(mx):
    """Two optimizers with their own control blocks and workspaces, interleaved on two streams."""
    def build(k):
        params, grads, _ = make(MIXED, [(200000,), (4097,)], 20 + k)
        clip = mx.GradClip(grads, max_norm=0.1 * (k + 1))
        return clip, mx.AdamWMulti(params, grads, state_bits=8, seed=k, control=clip.control)

    both, alone = [build(0), build(1)], [build(0), build(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (clip, opt), s in zip(both, streams):
            clip.step(stream=s)
            opt.step(stream=s)
    torch.cuda.synchronize()
    for clip, opt in alone:
        for _ in range(20):
            clip.step()
            opt.step()
        torch.cuda.synchronize()
    for (_, x), (_, y) in zip(both, alone):
        for p, q in zip(x.params, y.params):
            assert torch.equal(p, q)


def test_captured_step_replays_as_the_eager_one(mx):
    """Norm, clip and both state widths in one graph: each replay clips by its
    own gradients, counts its own step, and takes the lr factor of its time."""
    def build():
        params, grads, _ = make(MIXED, SIZES + [(50000,)], 31)
        clip = mx.GradClip(grads, max_norm=0.5, skip_nonfinite=True)
        return clip, mx.AdamWMulti(params, grads, lr=1e-2, weight_decay=0.1, seed=6, control=clip.control,
                                   state_bits=[8 if i % 2 else 32 for i in range(len(params))])

    (ce, eager), (cg, graphed) = build(), build()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cg.step()
        graphed.step()
    noise = torch.randn(1 << 20, device="cuda")
    for r in range(5):
        for grads in (eager.grads, graphed.grads):
            refill(grads, 60 + r)
            if r == 3:
                grads[2][0] = math.inf
        for c in (ce.control, cg.control):
            c.lr_factor.fill_(1.0 / (r + 1))
        ce.step()
        eager.step()
        graph.replay()
        noise.mul_(1.0001).add_(0.5)
        torch.cuda.synchronize()
        assert torch.equal(ce.control.block, cg.control.block), r
        assert int(cg.control.step) == (r + 1 if r < 3 else r)
        for p, q in zip(eager.params, graphed.params):
            assert torch.equal(p, q), r
        assert torch.equal(eager.codes_r.view(torch.uint8), graphed.codes_r.view(torch.uint8))
        assert torch.equal(eager.scales, graphed.scales) and torch.equal(eager.exp_avg_sq, graphed.exp_avg_sq)


def test_capture_without_control_is_refused_and_empty_lists_run(mx):
    p, g = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    opt = mx.AdamWMulti([p], [g])
    opt.step()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(RuntimeError, match="control"):
            opt.step()
    opt.step()
    torch.cuda.synchronize()
    assert opt.t == 2
    for bits in (8, 32):
        none = mx.AdamWMulti([p[:0], p[:0]], [g[:0], g[:0]], state_bits=bits)
        none.step()
        assert none.t == 1 and none.moments(0)[0].shape == (0,)


def test_moments_and_resume(mx, tmp_path):
    def build():
        params, grads, _ = make(MIXED, SIZES, 17)
        return mx.AdamWMulti(params, grads, lr=1e-2, seed=9, state_bits=[8 if i % 2 else 32 for i in range(len(params))])

    a = build()
    for t in range(4):
        refill(a.grads, 70 + t)
        a.step()
        if t == 1:
            torch.save({"opt": a.state_dict(), "params": [p.cpu() for p in a.params]}, tmp_path / "s.pt")
    saved = torch.load(tmp_path / "s.pt", weights_only=True)
    b = build()
    b.load_state_dict(saved["opt"])
    for p, q in zip(b.params, saved["params"]):
        p.copy_(q)
    for t in (2, 3):
        refill(b.grads, 70 + t)
        b.step()
    torch.cuda.synchronize()
    for i, (p, q) in enumerate(zip(a.params, b.params)):
        assert torch.equal(p, q)
        for x, y in zip(a.moments(i), b.moments(i)):
            assert x.shape == p.shape and torch.equal(x, y)
    m, v = a.moments(15)
    st = a._state(15)
    n = m.numel()
    s = st[2].double().cpu().numpy()
    assert np.allclose(f64(m), OM.code_value(codes(st[0])) * OM.per_block(s[:, 0], n), rtol=4 * U, atol=0)
    assert np.allclose(f64(v), (OM.code_value(codes(st[1])) * OM.per_block(s[:, 1], n)) ** 2, rtol=4 * U, atol=0)


def test_32_bit_states_agree_with_the_one_type_list(mx):
    """The same tensors through AdamW (one type a list, fp32 hyperparameters) and AdamWMulti."""
    params, grads, _ = make([(F32, F32)], [(5000,), (33,)], 2)
    twin = [p.clone() for p in params]
    one = mx.AdamW(twin, grads, lr=2.0 ** -7, betas=(0.875, 0.96875), eps=2.0 ** -20, weight_decay=0.125)  # exact in fp32
    many = mx.AdamWMulti(params, grads, lr=2.0 ** -7, betas=(0.875, 0.96875), eps=2.0 ** -20, weight_decay=0.125)
    for _ in range(3):
        one.step()
        many.step()
    torch.cuda.synchronize()
    for p, q in zip(params, twin):
        # three steps, each off by at most the roundings of check_step's bound on either side
        assert torch.all((p - q).abs() <= 3 * 2 * 20 * U * (q.abs() + 2.0 ** -6))


# ------------------------------------------------------------ with Muon

def muon_groups(seed):
    gen = torch.Generator().manual_seed(seed)
    shapes = [((2, 300, 700), BF16), ((3, 520, 256), BF16), ((1, 256, 128), F32)]
    return [((0.02 * torch.randn(s, generator=gen)).to(dt).cuda(), torch.randn(s, generator=gen).to(dt).cuda())
            for s, dt in shapes]


@pytest.mark.parametrize("compute", [0, 1])
def test_muon_under_a_control_block(mx, compute):
    """Scale 1 is the plain step bit for bit; a power of two is the plain step
    on gradients times it, bit for bit; skip changes nothing; lr_factor scales lr."""
    ga, gb = muon_groups(3), muon_groups(3)
    control = mx.StepControl("cuda")
    a = mx.MuonStep(ga, compute=compute, lr=0.01, weight_decay=0.1)
    b = mx.MuonStep(gb, compute=compute, lr=0.01, weight_decay=0.1, control=control)

    def same():
        torch.cuda.synchronize()
        for (w, _), (x, _) in zip(ga, gb):
            assert torch.equal(w, x)
        for m, n in zip(a.momentum_buffers, b.momentum_buffers):
            assert torch.equal(m, n)

    a.step()
    b.step()
    same()
    control.scale.fill_(0.25)
    for _, g in ga:
        g.mul_(0.25)
    a.step()
    b.step()
    same()
    control.skip.fill_(1)
    b.step()
    same()
    control.skip.fill_(0)
    control.lr_factor.fill_(0.5)
    a.lr = 0.005
    a.step()
    b.step()
    torch.cuda.synchronize()
    for (w, _), (x, _) in zip(ga, gb):
        # 1 - f*lr*wd is rounded once more, lr*s once more: one step of the weight's type, or 4u
        tol = 2.0 ** -7 if w.dtype == BF16 else 4 * U
        assert torch.all((w.double() - x.double()).abs() <= tol * w.double().abs() + 4 * U)


@pytest.mark.parametrize("bits", [32, 8])
def test_whole_model_step(mx, bits):
    """OptimizerStep with clipping, skipping and 8-bit states over a toy model,
    eager and captured: Muon matrices, embedding, head, norms, biases."""
    from oracle import oracle as O

    def build():
        gen = torch.Generator().manual_seed(21)
        spec = [("embed_tokens.weight", (96, 64), BF16), ("layers.0.attn.wq", (64, 64), F32), ("layers.0.attn.bias", (64,), F32),
                ("layers.0.mlp.up", (160, 64), F32), ("layers.0.norm.weight", (64,), BF16), ("lm_head.weight", (96, 64), F32),
                ("unused.weight", (64, 64), F32)]
        named = []
        for name, shape, dt in spec:
            p = (0.05 * torch.randn(shape, generator=gen)).to(dt).cuda()
            g = None if name.startswith("unused") else torch.randn(shape, generator=gen).to(dt).cuda()
            named.append((name, p, g))
        opt = mx.OptimizerStep(named, compute=mx.MUON_F32, muon_lr=0.02, muon_weight_decay=0.1, adam_lr=0.01,
                               adam_weight_decay=0.2, max_grad_norm=0.5, skip_nonfinite=True, adam_state_bits=bits, seed=1)
        return named, opt

    named, opt = build()
    (adam,) = opt.adamw
    assert sorted(set(adam.bits)) == sorted({32, bits})
    init = {n: f64(p) for n, p, _ in named}
    before = [snapshot(adam, i) for i in range(len(adam.params))]
    opt.step()
    torch.cuda.synchronize()
    norm, scale = OM.grad_norm([f64(g) for _, _, g in named if g is not None], 0.5)
    assert abs(float(opt.clip.control.norm) - norm) <= 2 * U * norm
    for i in range(len(adam.params)):
        check_step(adam, i, before[i], 1, scale=float(opt.clip.control.scale))
    for name, p, g in named:
        if g is None:
            assert np.array_equal(f64(p), init[name])
        elif opt.routing[name] == "muon":
            want = O.muon_step(init[name].reshape(p.shape), np.zeros(p.shape), scale * f64(g).reshape(p.shape), lr=0.02,
                               weight_decay=0.1)[0]
            assert O.relative_frobenius_error(f64(p).reshape(p.shape), want) <= 1e-5

    # captured: replays follow an eager twin, a bad step among them
    (ne, eager), (ng, graphed) = build(), build()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step()
    torch.cuda.current_stream().wait_stream(side)
    eager.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for r in range(4):
        for named_ in (ne, ng):
            refill([g for _, _, g in named_ if g is not None], 80 + r)
            if r == 2:
                named_[1][2][0, 0] = math.nan
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert int(graphed.clip.control.skip) == (r == 2)
        for (_, p, _), (_, q, _) in zip(ne, ng):
            assert torch.equal(p, q), r
    state = eager.state_dict()
    _, other = build()
    other.load_state_dict(state)
    assert int(other.clip.control.step) == int(eager.clip.control.step)
