"""CPU checks of the expert operators: what the C entry points and the torch
helpers refuse before anything is launched, and the C layer under sanitizers
with stand-in launchers (no GPU is touched here)."""

import os
import shutil
import subprocess

import pytest
import torch

import matrix_aware_optimizer_step_amd as mx
from matrix_aware_optimizer_step_amd import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_aware_optimizer_step_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "host_abi")
FAKE = 0x10000  # non-NULL, 16-byte aligned; never dereferenced: validation fails first
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
E4M3, F32, BF16, I32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32


def status_of(fn):
    with pytest.raises(L.MuonError) as e:
        fn()
    return e.value.status


def dense(rows=64, cols=200, count=1, ld=None, dtype=L.MUON_F32, base=FAKE, stride=None, ptrs=None, reserved=0):
    ld = cols if ld is None else ld
    return L.MuonBatch(ptrs, base, rows * ld if stride is None else stride, count, rows, cols, ld, dtype, reserved)


def codes(rows=64, cols=200, count=1, block_rows=1, ld=256, scale_ld=None, codes=FAKE, scales=FAKE, stride=None,
          scale_stride=None, reserved=0):
    high = -(-rows // block_rows)
    scale_ld = high if scale_ld is None else scale_ld
    return L.MuonCodes(codes, scales, rows * ld if stride is None else stride,
                       -(-cols // 128) * scale_ld if scale_stride is None else scale_stride, count, rows, cols, ld,
                       scale_ld, block_rows, reserved)


@pytest.mark.parametrize("bad", [
    dict(codes=None), dict(scales=None), dict(codes=FAKE + 8), dict(scales=FAKE + 2), dict(count=0), dict(count=70000),
    dict(rows=0), dict(cols=0), dict(block_rows=64), dict(ld=200), dict(ld=264), dict(ld=128), dict(ld=1 << 31),
    dict(scale_ld=63), dict(reserved=1), dict(count=2, stride=16), dict(count=2, scale_stride=5),
    dict(count=2, stride=64 * 256 + 8)])
def test_codes_are_checked(bad):
    good = codes()
    assert status_of(lambda: L.muon_block_quantize(dense(), None, None, 1, codes(**bad), None, 0)) == INVALID
    assert status_of(lambda: L.muon_block_matmul(codes(**bad), good, dense(64, 64), None, 0, 0, 0)) == INVALID
    assert status_of(lambda: L.muon_block_matmul(good, codes(**bad), dense(64, 64), None, 0, 0, 0)) == INVALID


def test_quantize_refuses():
    x, q, qt = dense(), codes(), codes(200, 64, ld=128)
    call = lambda x=x, pairs=None, weights=None, k=1, q=q, qt=None: L.muon_block_quantize(x, pairs, weights, k, q, qt, 0)
    assert status_of(lambda: call(q=None)) == INVALID                       # nothing to write
    assert status_of(lambda: call(x=dense(base=None))) == INVALID
    assert status_of(lambda: call(x=dense(base=FAKE + 2))) == INVALID
    assert status_of(lambda: call(x=dense(dtype=5))) == INVALID
    assert status_of(lambda: call(x=dense(ld=100))) == INVALID
    assert status_of(lambda: call(x=dense(rows=63))) == INVALID
    assert status_of(lambda: call(x=dense(cols=199))) == INVALID
    assert status_of(lambda: call(x=dense(count=2))) == INVALID
    assert status_of(lambda: call(qt=codes(200, 63, ld=128))) == INVALID    # not the transpose
    assert status_of(lambda: call(qt=codes(200, 64, ld=128, block_rows=128))) == INVALID
    assert status_of(lambda: call(k=2)) == INVALID                          # k without pairs
    assert status_of(lambda: call(weights=FAKE)) == INVALID
    assert status_of(lambda: call(pairs=FAKE, k=0)) == INVALID
    assert status_of(lambda: call(pairs=FAKE + 2)) == INVALID
    assert status_of(lambda: call(pairs=FAKE, weights=FAKE + 1)) == INVALID
    assert status_of(lambda: call(x=dense(ptrs=FAKE), pairs=FAKE)) == INVALID
    assert status_of(lambda: call(pairs=FAKE, q=codes(block_rows=128))) == UNSUPPORTED
    big = dict(rows=1 << 27, cols=1 << 20)
    assert status_of(lambda: call(x=dense(**big), q=codes(**big, ld=1 << 20))) == UNSUPPORTED


def test_matmul_refuses():
    a, b, c = codes(64), codes(100, block_rows=128), dense(64, 100)
    call = lambda a=a, b=b, c=c, offsets=None, product=0, add=0: L.muon_block_matmul(a, b, c, offsets, product, add, 0)
    assert status_of(lambda: call(a=codes(64, 100))) == INVALID             # columns differ
    assert status_of(lambda: call(c=dense(64, 99))) == INVALID
    assert status_of(lambda: call(c=dense(63, 100))) == INVALID
    assert status_of(lambda: call(a=codes(64, block_rows=128))) == UNSUPPORTED
    assert status_of(lambda: call(add=2)) == INVALID
    assert status_of(lambda: call(c=dense(64, 100, dtype=L.MUON_BF16), add=1)) == UNSUPPORTED
    assert status_of(lambda: call(product=3)) == INVALID
    assert status_of(lambda: call(offsets=FAKE)) == INVALID                 # offsets without segments
    assert status_of(lambda: call(a=codes(64, count=2))) == INVALID         # counts differ
    assert status_of(lambda: call(product=1)) == INVALID                    # no offsets
    assert status_of(lambda: call(product=1, offsets=FAKE + 2)) == INVALID
    assert status_of(lambda: call(product=1, offsets=FAKE, a=codes(64, count=2))) == INVALID
    assert status_of(lambda: call(product=1, offsets=FAKE, c=dense(64, 100, count=2))) == INVALID
    assert status_of(lambda: call(product=2, offsets=FAKE, b=codes(100, count=2))) == INVALID
    assert status_of(lambda: call(a=codes(64, ld=1 << 24), b=codes(100, ld=256))) == UNSUPPORTED
    wide = dict(rows=1 << 30, cols=100, ld=128)
    assert status_of(lambda: call(a=codes(**wide), b=codes(**wide), c=dense(1 << 30, 1 << 30))) == UNSUPPORTED


def route_desc(**kw):
    d = dict(logits=FAKE, ld=64, tokens=10, experts=64, k=4, dtype=L.MUON_F32, score=0, renormalize=1, groups=1,
             top_groups=1, group_best=2, align=1, scale=1.0)
    d.update(kw)
    return L.MuonRoute(*[d[n] for n, _ in L.MuonRoute._fields_])


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=FAKE + 2), dict(ld=63), dict(tokens=0), dict(tokens=1 << 31), dict(experts=513, ld=513),
    dict(k=0), dict(k=17), dict(k=65), dict(dtype=2), dict(score=2), dict(renormalize=2), dict(groups=0),
    dict(groups=33), dict(groups=7), dict(groups=8, top_groups=9), dict(groups=8, top_groups=0), dict(groups=32, k=3),
    dict(group_best=0), dict(group_best=3), dict(align=0), dict(align=1 << 17), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(tokens=1 << 30, k=4)])
def test_route_descriptions_are_checked(bad):
    r = route_desc(**bad)
    assert status_of(lambda: L.muon_route(r, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, 1 << 20, 0)) == INVALID
    assert status_of(lambda: L.muon_route_backward(r, FAKE, FAKE, FAKE, FAKE, 600, 0)) == INVALID


def test_route_refuses():
    need = L.muon_route_workspace(10, 64)
    call = lambda r=route_desc(), bias=None, chosen=FAKE, weights=FAKE, slots=FAKE, pairs=FAKE, offsets=FAKE, loads=None, \
        ws=FAKE, size=need: L.muon_route(r, bias, None, chosen, weights, slots, pairs, offsets, loads, ws, size, 0)
    assert status_of(lambda: call(chosen=None)) == INVALID
    assert status_of(lambda: call(weights=None)) == INVALID
    assert status_of(lambda: call(slots=None)) == INVALID       # all three or none
    assert status_of(lambda: call(offsets=None)) == INVALID
    for name in ("bias", "chosen", "weights", "slots", "loads"):
        assert status_of(lambda: call(**{name: FAKE + 2})) == INVALID
    assert status_of(lambda: call(ws=None)) == WORKSPACE
    assert status_of(lambda: call(size=need - 1)) == WORKSPACE
    assert status_of(lambda: call(ws=FAKE + 4)) == WORKSPACE
    assert status_of(lambda: call(r=route_desc(tokens=(1 << 29) - 1, k=1, experts=512, ld=512, align=1 << 16),
                                  size=1 << 40)) == UNSUPPORTED
    many = route_desc(tokens=(1 << 22) + 1)
    assert status_of(lambda: call(r=many, size=1 << 40)) == UNSUPPORTED  # an order, or loads alone, of too many tokens
    assert status_of(lambda: call(r=many, size=1 << 40, slots=None, pairs=None, offsets=None, loads=FAKE)) == UNSUPPORTED
    back = lambda chosen=FAKE, grad=FAKE, out=FAKE, ld=64: L.muon_route_backward(route_desc(), chosen, FAKE, grad, out, ld, 0)
    assert status_of(lambda: back(chosen=None)) == INVALID
    assert status_of(lambda: back(grad=None)) == INVALID
    assert status_of(lambda: back(out=FAKE + 2)) == INVALID
    assert status_of(lambda: back(ld=63)) == INVALID


def test_capacity_and_workspace():
    assert L.muon_route_capacity(10, 64, 4, 1) == 40
    assert L.muon_route_capacity(10, 64, 4, 128) == -(-(40 + 64 * 127) // 128) * 128
    assert L.muon_route_capacity(0, 64, 4, 1) == 0 == L.muon_route_capacity(10, 64, 65, 1)
    assert L.muon_route_capacity(1 << 22, 64, 4, 1) == 1 << 24 and L.muon_route_capacity((1 << 22) + 1, 64, 4, 1) == 0
    assert L.muon_route_workspace(0, 64) == 0 == L.muon_route_workspace(10, 513)
    assert L.muon_route_workspace(70, 100) == 5 * 112 and L.muon_route_workspace(1 << 20, 128) == (1 << 14) * 128


def test_balance_and_sums_refuse():
    call = lambda bias=FAKE, loads=FAKE, experts=64, rate=0.1, control=None: L.muon_balance_update(bias, loads, experts,
                                                                                                   rate, control, 0)
    for bad in (dict(bias=None), dict(loads=None), dict(bias=FAKE + 2), dict(experts=0), dict(experts=513),
                dict(rate=-1.0), dict(rate=float("nan")), dict(control=FAKE + 8)):
        assert status_of(lambda: call(**bad)) == INVALID
    y, out = dense(100, 64), dense(10, 64)
    total = lambda y=y, out=out, slots=FAKE, weights=None, k=4: L.muon_expert_sum(y, slots, weights, k, out, 0)
    dot = lambda y=y, grad=out, slots=FAKE, dots=FAKE, k=4: L.muon_expert_dot(grad, y, slots, k, dots, 0)
    for bad in (dict(slots=None), dict(slots=FAKE + 1), dict(k=0), dict(k=17), dict(y=dense(100, 63)),
                dict(y=dense(100, 64, count=2)), dict(y=dense(100, 64, base=None)), dict(y=dense(100, 64, ptrs=FAKE))):
        assert status_of(lambda: total(**bad)) == INVALID
        assert status_of(lambda: dot(**bad)) == INVALID
    assert status_of(lambda: total(weights=FAKE + 2)) == INVALID
    assert status_of(lambda: dot(dots=None)) == INVALID
    assert status_of(lambda: total(out=dense(1 << 30, 1 << 10, ld=1 << 10), y=dense(100, 1 << 10))) == UNSUPPORTED


# ------------------------------------------------------------ torch helpers, on the CPU

def block(rows, cols, block_rows=1, count=None):
    return mx.BlockCodes.empty(rows, cols, block_rows, count, "cpu")


def test_block_codes_take_what_fits():
    q = block(5, 200)
    assert q.codes.shape == (5, 200) and q.codes.stride() == (256, 1) and q.scales.shape == (2, 5)
    assert block(300, 128, 128, 2).scales.shape == (2, 1, 3)
    wide = torch.zeros(4, 256, dtype=torch.uint8).view(E4M3)
    mx.BlockCodes(wide[:, :130], torch.zeros(2, 4))
    mx.BlockCodes(wide[1:2, :130], torch.zeros(2, 1))
    for bad, kind in [
            (lambda: mx.BlockCodes(wide[:, :130], torch.zeros(4, 2)), ValueError),            # scales the other way round
            (lambda: mx.BlockCodes(wide.float()[:, :130], torch.zeros(2, 4)), TypeError),
            (lambda: mx.BlockCodes(wide[:, :130], torch.zeros(2, 4, dtype=BF16)), TypeError),
            (lambda: mx.BlockCodes(wide[:, :130], torch.zeros(2, 4), 64), ValueError),
            (lambda: mx.BlockCodes(wide.t(), torch.zeros(1, 256)), ValueError),
            (lambda: mx.BlockCodes(wide[:, :130], torch.zeros(4, 2).t()), ValueError),
            (lambda: mx.BlockCodes(wide[:, :130].clone(memory_format=torch.contiguous_format), torch.zeros(2, 4)),
             ValueError),                                                                     # rows not padded
            (lambda: mx.BlockCodes(wide.view(-1)[126:].as_strided((4, 130), (256, 1)), torch.zeros(2, 4)), ValueError),
            (lambda: mx.BlockCodes(wide[0], torch.zeros(2, 4)), ValueError)]:
        with pytest.raises(kind):
            bad()
    with pytest.raises(ValueError):
        q[0]


def test_quantize_checks_its_arguments():
    x = torch.zeros(6, 200)
    pairs, w = torch.zeros(9, dtype=I32), torch.zeros(6, 2)
    for bad in (dict(order="columns"), dict(block_rows=2), dict(weights=w), dict(pairs=pairs.long()),
                dict(pairs=pairs, block_rows=128), dict(pairs=pairs, weights=w[:5]), dict(pairs=pairs, weights=w.double()),
                dict(pairs=(pairs, 3), weights=w), dict(out=block(6, 199)), dict(out=(block(6, 200), block(6, 200)), order="both"),
                dict(pairs=pairs[::2])):
        with pytest.raises(ValueError):
            mx.quantize(x, **bad)
    with pytest.raises(ValueError):
        mx.quantize(torch.zeros(2, 6, 200), pairs=pairs)
    with pytest.raises(TypeError):
        mx.quantize(x.double())
    with pytest.raises(ValueError):
        mx.quantize(x.t())
    with pytest.raises(RuntimeError, match="no CPU path"):
        mx.quantize(x)


def test_products_check_their_arguments():
    a, b, b3 = block(6, 200), block(7, 200, 128), block(7, 200, 128, 3)
    o = torch.zeros(4, dtype=I32)
    for bad in (lambda: mx.block_matmul(a, block(7, 199)), lambda: mx.block_matmul(block(256, 200, 128), b),
                lambda: mx.block_matmul(a, b3), lambda: mx.block_matmul(a, b, out=torch.zeros(6, 8)),
                lambda: mx.block_matmul(a, b, accumulate=True), lambda: mx.block_matmul(a, b, out=torch.zeros(7, 6).t()),
                lambda: mx.expert_matmul(a, b, o), lambda: mx.expert_matmul(a, b3, o[:3]),
                lambda: mx.expert_matmul(a, b3, o.long()), lambda: mx.expert_grad(a, b3, o),
                lambda: mx.expert_grad(a, b, o, out=torch.zeros(3, 6, 8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mx.block_matmul(a, b, out=torch.zeros(6, 7, dtype=BF16), accumulate=True)
    with pytest.raises(TypeError):
        mx.block_matmul(a.codes, b)
    with pytest.raises(TypeError):
        mx.block_matmul(a, b, dtype=torch.float16)
    with pytest.raises(RuntimeError, match="no CPU path"):
        mx.block_matmul(a, b)


def test_routing_checks_its_arguments():
    z = torch.zeros(5, 40)
    for bad in (dict(k=0), dict(k=17), dict(k=41), dict(k=2, score="tanh"), dict(k=2, bias=torch.zeros(39)),
                dict(k=2, mask=torch.ones(4, dtype=torch.bool)), dict(k=2, loads=torch.zeros(39, dtype=I32)),
                dict(k=2, align=0)):
        with pytest.raises(ValueError):
            mx.route(z, **bad)
    for bad in (dict(bias=torch.zeros(40, dtype=BF16)), dict(mask=torch.ones(5)), dict(loads=torch.zeros(40))):
        with pytest.raises(TypeError):
            mx.route(z, 2, **bad)
    with pytest.raises(ValueError):
        mx.route(torch.zeros(5, 600), 2)
    with pytest.raises(ValueError):
        mx.route(torch.zeros(40, 5).t(), 2)
    with pytest.raises(TypeError):
        mx.route(z.half(), 2)
    with pytest.raises(RuntimeError, match="no CPU path"):
        mx.route(z, 2)
    r = mx.Routing(torch.zeros(5, 2, dtype=I32), torch.zeros(5, 2), None, None, None, "softmax", True, 1.0)
    for bad in (torch.zeros(5, 3), torch.zeros(2, 5).t()):
        with pytest.raises(ValueError):
            mx.route_backward(z, r, bad)
    with pytest.raises(ValueError):
        mx.route_backward(z, r, torch.zeros(5, 2), out=torch.zeros(5, 40, dtype=BF16))
    y, slots = torch.zeros(9, 16), torch.zeros(5, 2, dtype=I32)
    for bad in (lambda: mx.expert_sum(y, slots[0]), lambda: mx.expert_sum(y, slots, torch.zeros(5, 3)),
                lambda: mx.expert_sum(y, slots, out=torch.zeros(5, 15)), lambda: mx.expert_dot(torch.zeros(4, 16), y, slots),
                lambda: mx.expert_sum(y.t(), slots), lambda: mx.expert_sum(y, torch.zeros(5, 17, dtype=I32))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mx.expert_sum(y, slots.long())
    with pytest.raises(RuntimeError, match="no CPU path"):
        mx.expert_sum(y, slots)
    with pytest.raises(ValueError):
        mx.BalanceBias(0, device="cpu")


def test_balance_bias_state():
    a, b = mx.BalanceBias(8, 0.01, "cpu"), mx.BalanceBias(8, 0.5, "cpu")
    a.bias.copy_(torch.arange(8))
    a.loads.fill_(3)
    b.load_state_dict(a.state_dict())
    assert torch.equal(b.bias, a.bias) and torch.equal(b.loads, a.loads) and b.rate == 0.01
    with pytest.raises(ValueError):
        mx.BalanceBias(9, device="cpu").load_state_dict(a.state_dict())
    with pytest.raises(RuntimeError, match="no CPU path"):
        a.step()


def test_optimizer_step_checks_codes_and_balance():
    p = [("layers.0.w", torch.zeros(8, 8), torch.zeros(8, 8))]
    with pytest.raises(ValueError, match="no parameter named"):
        mx.OptimizerStep(p, codes={"w": ["layers.0.w", "layers.1.w"]})
    opt = mx.OptimizerStep(p, balance=[mx.BalanceBias(4, device="cpu")])
    state = opt.state_dict()
    opt.load_state_dict(state)
    plain = mx.OptimizerStep(p)
    assert plain.codes == {} and plain.balance == []
    with pytest.raises(ValueError, match="balance"):
        plain.load_state_dict(state)
    with pytest.raises(ValueError, match="balance"):
        opt.load_state_dict(plain.state_dict())


def test_abi_layer_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / "experts_sanitized"
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-Wall", "-Werror", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", CSRC, "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, "abi.cpp"),
           os.path.join(CSRC, "abi_experts.cpp"), os.path.join(HERE, "stub_launchers.cpp"),
           os.path.join(HERE, "experts_driver.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=env)
    assert out.returncode == 0, out.stderr[-4000:]
    assert out.stdout.startswith("ok: ")
