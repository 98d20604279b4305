"""GPU tests of the many-tensor operators' state at its edges: what lies behind
a tensor, restored states, streams that are being captured, descriptors that
the kernels pass over."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


SIZES = [300, 5, 256, 4097, 4096 + 250]


def build(mx, bits, control=None):
    gen = torch.Generator().manual_seed(4)
    types = [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)]
    params = [torch.randn(n, generator=gen).to(p).cuda() for n, (p, _) in zip(SIZES, types)]
    grads = [torch.randn(n, generator=gen).to(g).cuda() for n, (_, g) in zip(SIZES, types)]
    return mx.AdamWMulti(params, grads, lr=1e-2, state_bits=bits, seed=7, control=control)


def gaps(opt):
    """The state behind each tensor, up to the end of its last block."""
    out = []
    for i, p in enumerate(opt.params):
        end, n = opt._at[i] + p.numel(), -p.numel() % 256
        for buf in (opt.exp_avg, opt.exp_avg_sq) if opt.bits[i] == 32 else (opt.codes_m, opt.codes_r):
            out.append((buf.view(torch.uint8) if buf.element_size() == 1 else buf)[end:end + n])
    return out


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("through", ["gradient", "clip factor"])
def test_state_behind_a_tensor_stays_zero(mx, bits, bad, through):
    control = mx.StepControl("cuda", step=1)
    opt = build(mx, bits, control)
    opt.step()
    if through == "gradient":
        for g in opt.grads:
            g[-1] = bad
    else:
        control.scale.fill_(bad)
    for _ in range(3):
        opt.step()
    torch.cuda.synchronize()
    for gap in gaps(opt):
        assert torch.all(gap == 0)
    assert not math.isfinite(float(opt.moments(0)[0][-1]))  # the bad value did arrive


@pytest.mark.parametrize("bits", [8, 32])
def test_restoring_after_a_bad_step_resumes_bit_for_bit(mx, bits):
    """A state restored in place, after a step with a NaN, and one restored
    into a new object go on alike."""
    used = build(mx, bits)
    used.step()
    weights, saved = [p.clone() for p in used.params], used.state_dict()
    for g in used.grads:
        g[-1] = math.nan
    used.step()
    fresh = build(mx, bits)
    for opt in (used, fresh):
        for p, w in zip(opt.params, weights):
            p.copy_(w)
        for g, f in zip(opt.grads, build(mx, bits).grads):
            g.copy_(-f)  # the moments shrink: what is left behind a tensor would be its block's largest
        opt.load_state_dict(saved)
        for _ in range(3):
            opt.step()
    torch.cuda.synchronize()
    for i, (p, q) in enumerate(zip(used.params, fresh.params)):
        assert torch.equal(p, q)
        for x, y in zip(used._state(i), fresh._state(i)):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
