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


def table(obj, struct, count):
    """The descriptors of a list as int32 words in device memory, a row each."""
    import ctypes
    size = ctypes.sizeof(struct)
    (rows,) = [b for b in obj._buffers if b.data_ptr() == (obj.desc.params if hasattr(obj.desc, "params") else obj.desc.grads)]
    return rows[:count * size].view(torch.int32).view(count, size // 4)


@pytest.mark.parametrize("field,value", [("param_dtype", 2), ("param_dtype", -1), ("grad_dtype", 2), ("grad_dtype", 1 << 20),
                                         ("state_bits", 4), ("state_bits", 0)])
@pytest.mark.parametrize("bits", [8, 32])
def test_descriptors_of_no_type_are_left_alone(mx, field, value, bits):
    L = mx._lib
    opt, twin = build(mx, bits), build(mx, bits)
    table(opt, L.MuonParam, len(SIZES))[3, getattr(L.MuonParam, field).offset // 4] = value
    before = [opt.params[3].clone()] + [x.clone() for x in opt._state(3)]
    for o in (opt, twin):
        o.step()
    torch.cuda.synchronize()
    for x, y in zip(before, [opt.params[3]] + opt._state(3)):
        assert torch.equal(x.view(torch.uint8), y.contiguous().view(torch.uint8))
    for i in (0, 1, 2, 4):
        assert torch.equal(opt.params[i], twin.params[i])


@pytest.mark.parametrize("value", [2, -1, 1 << 20])
def test_gradients_of_no_type_add_nothing(mx, value):
    L = mx._lib
    grads = build(mx, 32).grads
    clip, rest = mx.GradClip(grads), mx.GradClip([g for i, g in enumerate(grads) if i != 3])
    table(clip, L.MuonGrad, len(grads))[3, L.MuonGrad.dtype.offset // 4] = value
    clip.step()
    rest.step()
    torch.cuda.synchronize()
    # the chunks go to workgroups in another grouping: two fp64 sums, rounded once
    assert abs(float(clip.control.norm) - float(rest.control.norm)) <= 2.0 ** -23 * float(rest.control.norm)


def test_only_the_calls_own_stream_decides_about_a_capture(mx):
    """Without a control block a step refuses a stream that is being captured,
    whichever stream is current, and takes one that is not."""
    opt, twin = build(mx, 8), build(mx, 8)
    captured, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = torch.zeros(64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=captured):
        keep.add_(1.0)
        opt.step(stream=other)
        with torch.cuda.stream(other):
            for stream in (captured, captured.cuda_stream):
                with pytest.raises(RuntimeError, match="control"):
                    opt.step(stream=stream)
            opt.step()
            opt.step(stream=other.cuda_stream)
        with pytest.raises(RuntimeError, match="control"):
            opt.step()
    assert opt.t == 3
    for _ in range(3):
        twin.step()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(opt.params, twin.params):
        assert torch.equal(p, q)


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 2.0 ** 125])
@pytest.mark.parametrize("bits", [8, 32])
def test_smallest_and_largest_eps(mx, bits, eps):
    """Elements that never had a gradient stay as they are, and the others
    follow m / (r + eps)."""
    n = 600
    p, g = torch.full((n,), 0.75, device="cuda"), torch.zeros(n, device="cuda")
    g[::3] = 2.0
    opt = mx.AdamWMulti([p], [g], lr=2.0 ** -4, betas=(0.5, 0.75), eps=eps, state_bits=bits)
    opt.step()
    torch.cuda.synchronize()
    # m = 1, v = 1, both corrected to 2 and 4: the step is 2^-4 * 2 / (2 + eps), with at most 8 roundings of its own
    want = 0.75 - 2.0 ** -4 * 2.0 / (2.0 + eps)
    assert torch.all((p[::3].double() - want).abs() <= 2.0 ** -24 * want + 8 * 2.0 ** -24 * 2.0 ** -4)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::3] = False
    assert torch.all(p[rest] == 0.75)


@pytest.mark.parametrize("explicit", [True, False])
def test_a_dropped_muon_step_outlives_its_kernels(mx, explicit):
    """MuonStep and its control block are dropped while the step still waits on
    a side stream: their memory must not go to new tensors before it ran."""
    gen = torch.Generator().manual_seed(2)
    g = torch.randn(2, 256, 320, generator=gen).cuda()
    w = torch.randn(2, 256, 320, generator=gen).cuda()
    twin = w.clone()
    mx.MuonStep([(twin, g)], lr=0.01, control=mx.StepControl("cuda")).step()
    step = mx.MuonStep([(w, g)], lr=0.01, control=mx.StepControl("cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        if not explicit:
            step.step()
    if explicit:
        step.step(stream=side)
    del step
    junk = [torch.full((n,), 2, dtype=torch.uint8, device="cuda") for n in [64] * 64 + [1 << 20] * 16]
    torch.cuda.synchronize()
    assert torch.equal(w, twin) and len(junk) == 80


def test_a_norm_past_the_largest_float(mx):
    """Finite gradients whose norm no float holds: an infinite norm, which
    counts as not finite, and a finite bound takes nothing of the gradients."""
    g = torch.full((3000,), 3e38, device="cuda")
    for max_norm, scale in ((1.0, 0.0), (math.inf, 1.0)):
        for skip in (False, True):
            c = mx.GradClip([g], max_norm=max_norm, skip_nonfinite=skip)
            c.step()
            c = c.control
            assert (float(c.norm), float(c.scale), int(c.skip), int(c.step)) == (math.inf, scale, skip, not skip)


def test_raw_handles_name_their_streams(mx):
    side = torch.cuda.Stream()
    for stream in (side, torch.cuda.default_stream()):
        assert mx.muon._stream_object(stream.cuda_stream).cuda_stream == stream.cuda_stream


def test_made_on_a_side_stream_and_stepped_on_the_default_one(mx):
    """By its handle, 0: the memory, the side stream's, outlives the step."""
    n = 1 << 20
    p, twin, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda"), torch.randn(n, device="cuda")
    mx.AdamWMulti([twin], [g], lr=1e-2).step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        opt = mx.AdamWMulti([p], [g], lr=1e-2)
    torch.cuda._sleep(50_000_000)
    opt.step(stream=0)
    del opt
    with torch.cuda.stream(side):
        junk = [torch.full((n,), 1e30, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(p, twin) and len(junk) == 8


def test_restored_values_are_there_for_any_stream(mx):
    """A load waits for its own device work, as the constructors do: a step on
    another stream right after it finds what was loaded."""
    g, side = torch.ones(300, device="cuda"), torch.cuda.Stream()
    counts = mx.StepControl("cuda", step=41).state_dict()
    clip = mx.GradClip([g])
    opt = mx.AdamWMulti([torch.ones(300, device="cuda")], [g], control=clip.control)
    saved = dict(opt.state_dict(), step=70)
    for load, step in ((lambda: clip.control.load_state_dict(counts), 42), (lambda: opt.load_state_dict(saved), 71)):
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        load()
        clip.step(stream=side)
        torch.cuda.synchronize()
        assert int(clip.control.step) == step
