"""CPU checks of the many-tensor operators' host side: what the Python classes
refuse, the tables they build, the C entry points' argument checks, and the
C-ABI layer under AddressSanitizer and UndefinedBehaviorSanitizer (nothing
touches a GPU)."""

import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_step_amd as mx
from matrix_aware_optimizer_step_amd import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_aware_optimizer_step_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "host_abi")
FAKE = 0x10000


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("params,grads,kw,error", [
    ([], [], {}, ValueError),
    ([z(3)], [], {}, ValueError),
    ([z(3)], [z(4)], {}, ValueError),
    ([z(3, dtype=torch.float16)], [z(3)], {}, TypeError),
    ([z(3)], [z(3, dtype=torch.float64)], {}, TypeError),
    ([z(4, 3).t()], [z(3, 4)], {}, ValueError),
    ([z(3, 4)], [z(4, 3).t()], {}, ValueError),
    ([z(3)], [z(3)], {"state_bits": 16}, ValueError),
    ([z(3)], [z(3)], {"state_bits": [8, 8]}, ValueError),
    ([z(3)], [z(3)], {"weight_decay": [0.1, 0.1]}, ValueError),
    ([z(3)], [z(3)], {"weight_decay": math.nan}, ValueError),
    ([z(3)], [z(3)], {"lr_factor": math.inf}, ValueError),
    ([z(3)], [z(3)], {"seed": -1}, ValueError),
    ([z(3)], [z(3)], {"seed": 1 << 32}, ValueError),
    ([z(3).to_sparse()], [z(3)], {}, RuntimeError),
    ([z(3)], [z(3).to_sparse()], {}, RuntimeError),
    ([z(3, dtype=torch.int32)], [z(3)], {}, TypeError),
])
def test_adamw_multi_refuses(params, grads, kw, error):
    with pytest.raises(error):
        mx.AdamWMulti(params, grads, **kw)


def test_adamw_multi_refuses_shared_memory():
    p = z(100)
    with pytest.raises(ValueError, match="overlap"):
        mx.AdamWMulti([p, p], [z(100), z(100)])           # a tied parameter listed twice
    with pytest.raises(ValueError, match="overlap"):
        mx.AdamWMulti([p[:60], p[50:]], [z(60), z(50)])
    with pytest.raises(ValueError, match="gradient overlaps"):
        mx.AdamWMulti([p], [p])
    with pytest.raises(ValueError, match="gradient overlaps"):
        mx.AdamWMulti([p[:40], p[60:]], [z(40), p[20:60]])  # another tensor's parameter
    mx.AdamWMulti([p[:50], p[50:], p[:0]], [z(50), z(50), z(0)])  # neighbours and an empty one are fine


@pytest.mark.parametrize("kw,error", [
    ({"max_norm": 0.0}, ValueError), ({"max_norm": -1.0}, ValueError), ({"max_norm": math.nan}, ValueError),
])
def test_grad_clip_refuses_bounds(kw, error):
    with pytest.raises(error):
        mx.GradClip([z(3)], **kw)


def test_grad_clip_refuses_tensors():
    for bad, error in (([], ValueError), ([z(3, dtype=torch.float16)], TypeError), ([z(4, 3).t()], ValueError),
                       ([z(3).to_sparse()], RuntimeError)):
        with pytest.raises(error):
            mx.GradClip(bad)
    with pytest.raises(ValueError):
        mx.StepControl("cpu", step=-1)


def test_calls_on_the_cpu_fail_before_the_library():
    """There is no CPU path: the tables build, the step does not run."""
    opt, clip = mx.AdamWMulti([z(3)], [z(3)]), mx.GradClip([z(3)])
    for call in (opt.step, clip.step, lambda: opt.step(stream=7), lambda: clip.step(stream=7)):
        with pytest.raises(RuntimeError, match="GPU"):
            call()
    assert opt.t == 0


def test_muon_step_refuses_a_control_it_cannot_follow():
    w, g, control = z(1, 64, 64), z(1, 64, 64), mx.StepControl("cpu")
    for kw in ({"packed": False}, {"fused_apply": True}, {"steps": 0}):
        with pytest.raises(ValueError):
            mx.MuonStep([(w, g)], control=control, **kw)
    with pytest.raises(ValueError):
        mx.OptimizerStep([("norm.weight", z(3), z(3))], adam_state_bits=4)


def test_tables_describe_the_tensors():
    sizes = [0, 5000, 4096, 1, 8193]
    params = [z(n, dtype=torch.bfloat16 if i % 2 else torch.float32) for i, n in enumerate(sizes)]
    grads = [z(n) for n in sizes]
    bits = [8, 8, 32, 8, 8]
    opt = mx.AdamWMulti(params, grads, weight_decay=[0.0, 0.1, 0.2, 0.3, 0.4], state_bits=bits)
    assert opt.desc.count == 5 and opt.desc.total_chunks == 0 + 2 + 1 + 1 + 3
    rows = (L.MuonParam * 5).from_address(opt.desc.params)
    chunk = (ctypes.c_int32 * 7).from_address(opt.desc.chunk_tensor)
    assert list(chunk) == [1, 1, 2, 3, 4, 4, 4]
    assert [r.first_chunk for r in rows] == [0, 0, 2, 3, 4]
    assert [r.counter for r in rows if r.state_bits == 8] == [0, 0, 5120, 5376]
    for i, r in enumerate(rows):
        assert (r.param or 0) == params[i].data_ptr() and (r.grad or 0) == grads[i].data_ptr() and r.numel == sizes[i]
        assert r.param_dtype == i % 2 and r.grad_dtype == 0 and r.weight_decay == np.float32(0.1 * i)
        assert r.m % 16 == 0 and r.v % 16 == 0
        if r.state_bits == 8:
            assert r.m == opt.codes_m.data_ptr() + r.counter and r.scales == opt.scales.data_ptr() + r.counter // 256 * 8
        else:
            assert r.m == opt.exp_avg.data_ptr() and r.scales is None
    assert opt.codes_m.numel() == 5120 + 256 + 8448 and tuple(opt.scales.shape) == ((5120 + 256 + 8448) // 256, 2)
    clip = mx.GradClip([z(16384), z(0), z(16385, dtype=torch.bfloat16)])
    assert clip.desc.total_chunks == 3 and list((ctypes.c_int32 * 3).from_address(clip.desc.chunk_tensor)) == [0, 2, 2]
    assert [g.dtype for g in (L.MuonGrad * 3).from_address(clip.desc.grads)] == [0, 0, 1]


def test_state_dict_round_trip_and_mismatch():
    a = mx.AdamWMulti([z(300), z(5)], [z(300), z(5)], state_bits=[8, 32], seed=3)
    a.codes_m.view(torch.uint8).copy_(torch.arange(512) % 120)
    a.scales.fill_(0.5)
    a.t = 7
    b = mx.AdamWMulti([z(300), z(5)], [z(300), z(5)], state_bits=[8, 32])
    b.load_state_dict(a.state_dict())
    assert b.t == 7 and b.seed == 3 and b.hyper.seed == 3
    assert torch.equal(b.moments(0)[0], a.moments(0)[0]) and b.moments(0)[0].shape == (300,)
    for other in (mx.AdamWMulti([z(301), z(5)], [z(301), z(5)], state_bits=[8, 32]),
                  mx.AdamWMulti([z(300), z(5)], [z(300), z(5)], state_bits=32),
                  mx.AdamWMulti([z(300)], [z(300)], state_bits=8)):
        with pytest.raises(ValueError):
            other.load_state_dict(a.state_dict())
    one_type = mx.AdamW([z(300), z(5)], [z(300), z(5)])
    with pytest.raises(ValueError):
        b.load_state_dict(one_type.state_dict())


def test_control_block_layout():
    c = mx.StepControl("cpu", step=5)
    assert ctypes.sizeof(L.MuonStepControl) == 64 and c.block.numel() == 64
    raw = L.MuonStepControl.from_address(c.data_ptr())
    assert (raw.scale, raw.lr_factor, raw.step, raw.skip, raw.skipped) == (1.0, 1.0, 5, 0, 0)
    c.lr_factor.fill_(0.25)
    assert raw.lr_factor == 0.25


def status_of(fn):
    with pytest.raises(L.MuonError) as e:
        fn()
    return e.value.status


def test_entry_points_refuse_bad_arguments():
    grads, params = L.MuonGradList(1, 1, FAKE, FAKE), L.MuonParamList(1, 1, FAKE, FAKE)
    hyper = L.MuonAdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0, 0)
    ws = L.muon_grad_norm_workspace(1)
    assert status_of(lambda: L.muon_grad_norm(grads, 0.0, 0, FAKE, FAKE, ws, 0)) == 1
    assert status_of(lambda: L.muon_grad_norm(grads, 1.0, 0, FAKE, FAKE, ws - 1, 0)) == 3
    assert status_of(lambda: L.muon_grad_norm(L.MuonGradList(0, 1, FAKE, FAKE), 1.0, 0, FAKE, FAKE, ws, 0)) == 1
    assert status_of(lambda: L.muon_adamw_multi(params, hyper, 0, None, 0)) == 1
    hyper.beta2 = 1.0
    assert status_of(lambda: L.muon_adamw_multi(params, hyper, 1, None, 0)) == 1


def test_abi_layer_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / "optim_sanitized"
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-Wall", "-Werror", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", CSRC, "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, "abi.cpp"),
           os.path.join(CSRC, "abi_optim.cpp"), os.path.join(HERE, "stub_launchers.cpp"),
           os.path.join(HERE, "optim_stubs.cpp"), os.path.join(HERE, "optim_driver.cpp"), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=env)
    assert out.returncode == 0, out.stderr[-4000:]
    assert out.stdout.startswith("ok: ")
