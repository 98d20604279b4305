"""CPU checks of what the many-tensor operators save, restore and refuse on the
host (nothing touches a GPU)."""

import os
import shutil
import subprocess

import pytest
import torch

import matrix_aware_optimizer_step_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_aware_optimizer_step_amd", "csrc")


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def raw(buffer):
    return buffer.view(torch.uint8) if buffer.element_size() == 1 else buffer


def buffers(opt):
    return [raw(b) for b in (opt.exp_avg, opt.exp_avg_sq, opt.codes_m, opt.codes_r)]


def test_load_clears_what_lies_behind_the_tensors():
    """The state is padded to whole blocks, and a block's maximum is taken over
    its padding too: nothing there may outlive a load."""
    def build():
        return mx.AdamWMulti([z(300), z(5), z(1)], [z(300), z(5), z(1)], state_bits=[8, 32, 8])

    a, b = build(), build()
    a.codes_m.view(torch.uint8)[:300] = 0x30
    a.exp_avg[:5] = 2.0
    for buf in buffers(b):
        buf.fill_(0xFE if buf.dtype == torch.uint8 else float("nan"))
    b.scales.fill_(float("nan"))
    b.load_state_dict(a.state_dict())
    for x, y in zip(buffers(a), buffers(b)):
        assert torch.equal(x, y)
    assert torch.equal(a.scales, b.scales)


def muon(control=None, **kw):
    w, g = z(1, 64, 64), z(1, 64, 64)
    return mx.MuonStep([(w, g)], control=control, **kw)


def test_muon_step_refuses_a_control_block_on_another_device():
    muon(mx.StepControl("cpu"))
    block = mx.StepControl("cpu")
    for elsewhere in ("cuda:0", "meta"):
        block.device = torch.device(elsewhere)
        with pytest.raises(ValueError, match="another device"):
            muon(block)


class Recorded:
    """Stands in for a library call and keeps its arguments."""

    def __init__(self, log, name):
        self.log, self.name = log, name

    def __call__(self, *args):
        self.log.append((self.name, args))


@pytest.fixture
def calls(monkeypatch):
    """MuonStep's library calls, recorded in order, on no device."""
    from matrix_aware_optimizer_step_amd import muon as mu
    log = []
    for name in ("muon_momentum_packed_grouped", "muon_momentum_packed_grouped_controlled",
                 "muon_orthogonalize_packed_grouped", "muon_orthogonalize_apply_packed_grouped", "muon_apply_grouped",
                 "muon_apply_grouped_controlled"):
        monkeypatch.setattr(mu.L, name, Recorded(log, name))
    return log


def test_muon_step_checks_its_path_before_every_step(calls):
    """The folded apply does not follow a control block, also when it is asked
    for after construction."""
    step = muon(mx.StepControl("cpu"))
    step.step(stream=7)
    assert [name for name, _ in calls] == ["muon_momentum_packed_grouped_controlled", "muon_orthogonalize_packed_grouped",
                                           "muon_apply_grouped_controlled"]
    calls.clear()
    for name, value in (("fused_apply", True), ("packed", False), ("steps", 0)):
        old = getattr(step, name)
        setattr(step, name, value)
        with pytest.raises(ValueError, match="control block"):
            step.step(stream=7)
        setattr(step, name, old)
    assert calls == []


FORMS = """
#include <cstdio>
#include "muon_internal.h"
int main() {
  const int bits[] = {-8, 0, 1, 4, 8, 16, 31, 32, 33, 64, 264};
  const int types[] = {-2147483647, -1, 0, 1, 2, 3, 4, 256, 2147483647};
  for (int b : bits)
    for (int p : types)
      for (int g : types) std::printf("%d %d %d %d\\n", b, p, g, muon::param_form(b, p, g));
  for (int g : types) std::printf("%d %d\\n", g, muon::known_type(g));
}
"""


def test_only_the_eight_forms_are_taken(tmp_path):
    """A type code or a state width that is none never picks a form (a 32-bit
    tensor has no scales for the 8-bit form to read)."""
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    (tmp_path / "forms.cpp").write_text(FORMS)
    exe = tmp_path / "forms"
    res = subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", CSRC,
                          str(tmp_path / "forms.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    lines = [tuple(map(int, line.split())) for line in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split("\n") if line]
    assert len(lines) == 11 * 9 * 9 + 9
    seen = set()
    for row in lines:
        if len(row) == 2:
            assert row[1] == (row[0] in (0, 1)), row
            continue
        bits, p, g, form = row
        if bits in (8, 32) and p in (0, 1) and g in (0, 1):
            assert form == (4 if bits == 8 else 0) + 2 * p + g, row
            seen.add(form)
        else:
            assert form == -1, row
    assert seen == set(range(8))


def test_adamw_multi_refuses_more_chunks_than_one_launch_holds():
    """A launch has fewer than 2^32 work-items, 256 of them to a chunk."""
    L = mx._lib
    hyper = L.MuonAdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0, 0)
    for chunks in (1 << 24, (1 << 31) - 1, 1 << 31):
        with pytest.raises(L.MuonError, match="total_chunks") as e:
            L.muon_adamw_multi(L.MuonParamList(1, chunks, 0x10000, 0x10000), hyper, 1, None, 0)
        assert e.value.status == 1


@pytest.mark.parametrize("eps", [2.0 ** -149, 1e-40, 2.0 ** -126 * (1 - 2.0 ** -24), 2.0 ** 125 * (1 + 2.0 ** -23), 1e39])
def test_adamw_multi_refuses_an_eps_that_its_reciprocal_loses(eps):
    """The hardware's reciprocal of a denominator below 2^-126 is infinite, and
    above 2^126 zero."""
    L = mx._lib
    with pytest.raises(L.MuonError, match="eps") as e:
        L.muon_adamw_multi(L.MuonParamList(1, 1, 0x10000, 0x10000), L.MuonAdamWHyper(1e-3, 0.9, 0.999, eps, 0, 0), 1, None, 0)
    assert e.value.status == 1


MODEL = [("embed_tokens.weight", (24, 16)), ("layers.0.attn.wq", (16, 16)), ("layers.0.norm.weight", (16,))]
MUON_ONLY = [("layers.0.attn.wq", (16, 16)), ("layers.0.attn.wk", (16, 16))]


def model_step(spec, **kw):
    return mx.OptimizerStep([(name, z(*shape), z(*shape)) for name, shape in spec], **kw)


@pytest.mark.parametrize("spec", [MODEL, MUON_ONLY])
def test_a_whole_step_saves_its_control_block(spec, tmp_path):
    a, b = model_step(spec, max_grad_norm=1.0), model_step(spec, max_grad_norm=1.0)
    a.clip.control.step.fill_(41)
    a.clip.control.skipped.fill_(3)
    a.clip.control.lr_factor.fill_(0.25)
    torch.save(a.state_dict(), tmp_path / "s.pt")
    b.load_state_dict(torch.load(tmp_path / "s.pt", weights_only=True))
    c = b.clip.control
    assert (int(c.step), int(c.skipped), float(c.lr_factor)) == (41, 3, 0.25)


def test_states_with_and_without_a_control_block():
    """A step without clipping takes a clipped one's state, and the reverse
    keeps the block's lr factor; so does a state saved without the block."""
    clipped, plain = model_step(MODEL, max_grad_norm=1.0, adam_state_bits=8), model_step(MODEL, adam_state_bits=8)
    clipped.clip.control.step.fill_(9)
    plain.load_state_dict(clipped.state_dict())
    assert plain.adamw[0].t == 9
    clipped.clip.control.lr_factor.fill_(0.5)
    plain.adamw[0].t = 12
    clipped.load_state_dict(plain.state_dict())
    assert int(clipped.clip.control.step) == 12 and float(clipped.clip.control.lr_factor) == 0.5
    old = clipped.state_dict()
    del old["control"]
    clipped.clip.control.step.fill_(0)
    clipped.load_state_dict(old)
    assert int(clipped.clip.control.step) == 12


def test_a_control_block_by_itself():
    a, b = mx.StepControl("cpu", step=5), mx.StepControl("cpu")
    a.lr_factor.fill_(0.125)
    a.skipped.fill_(2)
    b.load_state_dict(a.state_dict())
    assert (int(b.step), int(b.skipped), float(b.lr_factor)) == (5, 2, 0.125)


def test_a_refused_state_changes_nothing():
    """Every part is checked before any is copied, whichever does not fit."""
    one_type, many = model_step(MODEL[1:]), model_step(MODEL[1:], max_grad_norm=1.0)
    for own, other in ((one_type, many), (many, one_type)):
        other.muon.momentum_buffers[0].fill_(3.0)
        own.muon.lr = 0.75
        with pytest.raises(ValueError, match="saved for"):
            own.load_state_dict(other.state_dict())
        assert torch.all(own.muon.momentum_buffers[0] == 0.0) and own.muon.lr == 0.75
        other.muon.momentum_buffers[0].zero_()
    bad = many.state_dict()
    bad["control"] = {"step": 7}
    many.muon.momentum_buffers[0].fill_(5.0)
    with pytest.raises(ValueError, match="saved for"):
        many.load_state_dict(bad)
    assert torch.all(many.muon.momentum_buffers[0] == 5.0)
    bad = many.state_dict()
    bad["muon"]["momentum"][0] = z(1, 16, 17)
    many.clip.control.step.fill_(4)
    many.adamw[0].exp_avg.fill_(2.0)
    with pytest.raises(ValueError, match="saved for"):
        many.load_state_dict(bad)
    assert int(many.clip.control.step) == 4 and torch.all(many.adamw[0].exp_avg == 2.0)


def test_muon_step_holds_its_memory_on_every_stream(calls, monkeypatch):
    """What a MuonStep allocated, and the control block it reads, are recorded
    once on each stream that its kernels go to."""
    from matrix_aware_optimizer_step_amd import muon as mu
    log = []
    monkeypatch.setattr(mu, "_record_on", lambda s, ts: log.append((s, [t.data_ptr() for t in ts])))
    for name in ("muon_momentum_grouped", "muon_orthogonalize_grouped"):
        monkeypatch.setattr(mu.L, name, Recorded(calls, name))
    control = mx.StepControl("cpu")
    step = mx.MuonStep([([z(16, 16), z(16, 16)], [z(16, 16), z(16, 16)]), (z(1, 8, 8), z(1, 8, 8))], control=control)
    for stream in (7, 7, 8, 7):
        step.step(stream=stream)
    assert [s for s, _ in log] == [7, 8]
    mine = [control.block, *step.momentum_buffers, *step.ortho_buffers, *step.sumsq_buffers, *step.pws,
            *(t for b in step.w + step.g for t in b.owned)]
    assert len(mine) == 1 + 3 * 2 + 1 + 2
    assert all(sorted(ptrs) == sorted(t.data_ptr() for t in mine) for _, ptrs in log)
    # buffers made by a later step are recorded too
    log.clear()
    folded = mx.MuonStep([(z(1, 16, 16), z(1, 16, 16))], fused_apply=True)
    folded.step(stream=7)
    folded.packed = False
    folded.step(stream=7)
    assert [s for s, _ in log] == [7, 7]
    late = [*(b.keep[0] for b in folded.n + folded.o), *folded.mws, *folded.ows]
    assert len(late) == 4 and {t.data_ptr() for t in late} <= set(log[1][1])


def test_muon_step_runs_on_its_own_device(calls, monkeypatch):
    """The norm goes to its tensors' device whichever is current; Muon under
    the same block has to follow it there, onto that device's stream."""
    import contextlib
    current = [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    class Stream:
        def __init__(self, index):
            self.cuda_stream = 100 + index

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(current[0]))
    monkeypatch.setattr(mx.muon, "_record_on", lambda *a: None)
    step = muon(mx.StepControl("cpu"))
    step.device = torch.device("cuda:1")  # the library's calls are stand-ins
    for now in (0, 1):
        current[0] = now
        calls.clear()
        step.step()
        assert len(calls) == 3 and all(args[-1] == 101 for _, args in calls)
        assert current[0] == now


def test_hyperparameters_set_between_steps_reach_the_next(monkeypatch):
    opt = mx.AdamWMulti([z(300)], [z(300)], state_bits=8, seed=3)
    seen = []
    monkeypatch.setattr(opt, "_on", lambda stream: 0)
    monkeypatch.setattr(opt, "_capturing", lambda *a: False)
    monkeypatch.setattr(mx._lib, "muon_adamw_multi", lambda desc, h, *a: seen.append((h.lr, h.beta1, h.beta2, h.eps, h.seed)))
    opt.step()
    opt.lr, opt.betas, opt.eps, opt.seed = 0.5, (0.25, 0.75), 1e-6, 9
    opt.step()
    assert seen == [(1e-3, 0.9, 0.999, 1e-8, 3), (0.5, 0.25, 0.75, 1e-6, 9)] and opt.t == 2


def test_the_handle_zero_is_the_default_stream(monkeypatch):
    """ExternalStream(0) is a new stream of torch's own, not the default one."""
    default = object()
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, *a: ("external", raw))
    assert mx.muon._stream_object(0) is default
    assert mx.muon._stream_object(7) == ("external", 7)
