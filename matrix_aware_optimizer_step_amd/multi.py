"""Many-tensor operators of libmuon355 for torch: the gradient norm with its
clip factor and step count, and AdamW over tensors of any types with 32-bit or
8-bit moments ("LLM Optimizers: From SGD and AdamW to SOAP, Muon, and Scalable
Training", sections 5 and 6).

A ``StepControl`` is the device-side link between them: ``GradClip.step()``
writes the norm, the clip factor, the skip flag and the step count there, and
``AdamWMulti.step()`` (and ``MuonStep`` with ``control=``) read them when their
kernels run.  Nothing comes back to the host in between, so a whole clipped
step can be captured in a graph, and each replay clips by its own gradients
and counts its own steps.
"""

from __future__ import annotations

import bisect
import ctypes
import math

import numpy as np
import torch

from . import _lib as L
from .muon import _stream, _stream_object, dtype_code, workspace

# The raw handle of the current stream without a Stream object around it
# (1.7 us less in a call that takes 6); the public way where torch lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: int(torch.cuda.current_stream(index).cuda_stream))

MAX_POSITIONS = 1 << 36  # positions of the 8-bit states' random bits: 2^32 groups of 16 elements


def _device_of(device) -> torch.device:
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _check_dense(t: torch.Tensor, what: str) -> None:
    if t.is_sparse:
        raise RuntimeError("dense gradients required")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    dtype_code(t)  # bfloat16 or float32


def _check_apart(params, grads) -> None:
    """No parameter shares memory with another or with a gradient: all are
    updated in one launch."""
    def spans(tensors):
        return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t.numel()]

    written = sorted(spans(params))
    for (_, end), (start, _) in zip(written, written[1:]):
        if end > start:
            raise ValueError("two parameters overlap in memory (list a tied parameter once)")
    starts = [a for a, _ in written]
    for a, b in spans(grads):
        k = bisect.bisect_left(starts, b) - 1  # the last parameter that starts before the gradient's end
        if k >= 0 and written[k][1] > a:
            raise ValueError("a gradient overlaps a parameter in memory")


def _settle(device) -> None:
    """What the current stream wrote is there: any stream may use it from here on."""
    if device.type == "cuda":
        torch.cuda.current_stream(device).synchronize()


def _table(structs, device) -> torch.Tensor:
    """An array of ctypes structures in device memory."""
    return torch.from_numpy(np.frombuffer(bytes(structs), dtype=np.uint8).copy()).to(device)


def _chunks(numels, chunk):
    """(first chunk of each tensor, tensor of each chunk)."""
    per = [-(-n // chunk) for n in numels]
    first = [0]
    for n in per:
        first.append(first[-1] + n)
    return first, np.repeat(np.arange(len(numels), dtype=np.int32), per)


class _OnDevice:
    """Buffers made once for one device, and the stream each call goes to."""

    def _own(self, device, buffers) -> None:
        self.device = device
        self._buffers = [b for b in buffers if b is not None]
        self._seen = set()  # streams that the allocator knows these buffers are used on
        _settle(device)
        if device.type == "cuda":
            self._seen.add(_raw_stream(device.index))

    def _on(self, stream):
        """Raw stream of a call (None: the current one).  A stream other than
        the one the buffers were made on is recorded on them once, so that
        their memory outlives its kernels."""
        if self.device.type != "cuda":
            raise RuntimeError("the tensors are not on a GPU (there is no CPU path)")
        raw = _raw_stream(self.device.index) if stream is None else _stream(stream)
        if raw not in self._seen:
            with torch.cuda.device(self.device):  # a raw handle is a stream of the current device
                used = torch.cuda.current_stream() if stream is None else _stream_object(stream)
                for b in self._buffers:
                    b.record_stream(used)
            self._seen.add(raw)
        return raw

    def _here(self) -> bool:
        """Whether this object's device is current (asked once a call)."""
        return self.device.type != "cuda" or self.device.index == torch.cuda.current_device()

    def _capturing(self, stream, here: bool) -> bool:
        """Whether the stream of a call (None: the current one) is being captured."""
        if stream is None and here:
            return torch.cuda.is_current_stream_capturing()
        with torch.cuda.device(self.device):
            with torch.cuda.stream(torch.cuda.current_stream() if stream is None else _stream_object(stream)):
                return torch.cuda.is_current_stream_capturing()

    def _call(self, here: bool, fn, *args) -> None:
        """Runs fn with this object's device current."""
        if here:
            fn(*args)
        else:
            with torch.cuda.device(self.device):
                fn(*args)


class StepControl:
    """One step's control block in device memory (muon_step_control_t).

    ``norm``, ``scale``, ``skip``, ``step`` and ``skipped`` are 0-dim views:
    reading them with ``.item()`` waits for the device, using them in further
    device work does not.  ``lr_factor`` multiplies the learning rate of every
    call that reads the block; write it with ``lr_factor.fill_(x)``, also
    between replays of a captured step.  Calls that share a block must be
    ordered: on one stream, or by events.
    """

    def __init__(self, device="cuda", step: int = 0):
        if step < 0:
            raise ValueError("step counts updates from 0")
        self.device = _device_of(device)
        self.block = torch.zeros(ctypes.sizeof(L.MuonStepControl), dtype=torch.uint8, device=self.device)
        f32, i32, i64 = self.block.view(torch.float32), self.block.view(torch.int32), self.block.view(torch.int64)
        at = {name: getattr(L.MuonStepControl, name).offset for name, _ in L.MuonStepControl._fields_}
        self.norm, self.scale, self.lr_factor = f32[at["norm"] // 4], f32[at["scale"] // 4], f32[at["lr_factor"] // 4]
        self.skip = i32[at["skip"] // 4]
        self.step, self.skipped = i64[at["step"] // 8], i64[at["skipped"] // 8]
        self.scale.fill_(1.0)
        self.lr_factor.fill_(1.0)
        self.step.fill_(step)
        _settle(self.device)

    def data_ptr(self) -> int:
        return self.block.data_ptr()

    def state_dict(self) -> dict:
        """What the next step goes on from: both counts and the lr factor."""
        return {"step": int(self.step.item()), "skipped": int(self.skipped.item()),
                "lr_factor": float(self.lr_factor.item())}

    def check_state(self, state: dict) -> None:
        """Raises where load_state_dict() would refuse the state."""
        if not {"step", "skipped", "lr_factor"} <= set(state):
            raise ValueError("the state was saved for something else than a control block")

    def load_state_dict(self, state: dict) -> None:
        self.check_state(state)
        self.step.fill_(int(state["step"]))
        self.skipped.fill_(int(state["skipped"]))
        self.lr_factor.fill_(float(state["lr_factor"]))
        _settle(self.device)


class GradClip(_OnDevice):
    """Global norm of a list of gradients, and the factor that clips it.

    ``grads``: dense, contiguous bfloat16 and float32 tensors in any mix, read
    from the same storage at every step.  ``step()`` enqueues
    ``muon_grad_norm``: it writes norm, min(1, max_norm / norm) and the step
    count to ``control`` and leaves the gradients as they are; the updates that
    share the control block apply the factor as they read them.  With
    ``skip_nonfinite`` a norm that is not finite makes those updates leave
    everything unchanged, and the step is not counted.  ``max_norm`` may be
    infinity (count and check only).
    """

    def __init__(self, grads, *, max_norm: float = 1.0, skip_nonfinite: bool = False, control: StepControl | None = None):
        grads = list(grads)
        if not grads:
            raise ValueError("no gradients")
        device = grads[0].device
        for g in grads:
            _check_dense(g, "gradients")
            if g.device != device:
                raise ValueError("all gradients must be on one device")
        if not max_norm > 0:
            raise ValueError("max_norm must be > 0")
        if control is None:
            control = StepControl(device)
        if control.device != device:
            raise ValueError("control is on another device than the gradients")
        self.grads, self.control = grads, control
        self.max_norm, self.skip_nonfinite = float(max_norm), bool(skip_nonfinite)
        first, chunk_tensor = _chunks([g.numel() for g in grads], L.GRAD_CHUNK)
        tensors = _table((L.MuonGrad * len(grads))(*[
            L.MuonGrad(g.data_ptr(), g.numel(), first[i], dtype_code(g), 0) for i, g in enumerate(grads)]), device)
        chunks = torch.from_numpy(chunk_tensor).to(device)
        self.ws = workspace(L.muon_grad_norm_workspace(first[-1]), device)
        self.desc = L.MuonGradList(len(grads), first[-1], tensors.data_ptr(), chunks.data_ptr())
        self._own(device, [tensors, chunks, self.ws, control.block])

    def step(self, stream=None) -> None:
        raw = self._on(stream)
        self._call(self._here(), L.muon_grad_norm, self.desc, self.max_norm,
                   L.SKIP_NONFINITE if self.skip_nonfinite else 0, self.control.data_ptr(), self.ws.data_ptr(),
                   self.ws.numel(), raw)


def _per_tensor(x, n, what):
    out = list(x) if isinstance(x, (list, tuple)) else [x] * n
    if len(out) != n:
        raise ValueError(f"{what} needs one value, or one for each parameter")
    return out


class AdamWMulti(_OnDevice):
    """AdamW over any number of tensors of any types in one launch.

    ``params`` and ``grads``: lists of dense, contiguous tensors of matching
    shapes, bfloat16 or float32 each; the gradients are read from the same
    storage at every step.  ``weight_decay``, ``lr_factor`` (multiplies ``lr``)
    and ``state_bits`` are one value, or one for each parameter.

    ``state_bits=32`` keeps fp32 moments.  ``state_bits=8`` keeps m and
    r = sqrt(v) as e4m3 codes with one fp32 scale each per 256 elements (a
    quarter of the memory, less than half of the bytes a step moves), rounded
    stochastically by bits that depend on ``seed``, the step number and the
    element's position alone; muon355.h gives the format.

    With ``control`` the gradients' clip factor, the skip flag, the step number
    and the lr factor are read on the device (see ``StepControl``): run the
    ``GradClip`` that shares it before each step.  Otherwise ``t`` counts the
    steps, and a step cannot be captured (every replay would repeat its t).

    State buffers, each tensor starting on a multiple of 256 elements: ``exp_avg`` and
    ``exp_avg_sq`` (fp32) of the 32-bit tensors, ``codes_m``, ``codes_r``
    (float8_e4m3fn) and ``scales`` ([blocks, 2]: of m, of r) of the 8-bit ones;
    None where no tensor has that width.  ``moments(i)`` gives (m, v) of tensor
    i as fp32.
    """

    def __init__(self, params, grads, *, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0,
                 lr_factor=1.0, state_bits=32, seed: int = 0, control: StepControl | None = None):
        params, grads = list(params), list(grads)
        if not params or len(params) != len(grads):
            raise ValueError("need matching, non-empty lists of parameters and gradients")
        device = params[0].device
        n = len(params)
        for p, g in zip(params, grads):
            if p.shape != g.shape:
                raise ValueError("parameter and gradient shapes differ")
            _check_dense(p, "parameters")
            _check_dense(g, "gradients")
            if p.device != device or g.device != device:
                raise ValueError("all tensors must be on one device")
        _check_apart(params, grads)
        if control is not None and control.device != device:
            raise ValueError("control is on another device than the parameters")
        if not 0 <= int(seed) < 1 << 32:
            raise ValueError("seed outside [0, 2^32)")
        decays = [float(x) for x in _per_tensor(weight_decay, n, "weight_decay")]
        factors = [float(x) for x in _per_tensor(lr_factor, n, "lr_factor")]
        bits = _per_tensor(state_bits, n, "state_bits")
        if not all(map(math.isfinite, decays + factors)):
            raise ValueError("weight_decay and lr_factor must be finite")
        if any(b not in (8, 32) for b in bits):
            raise ValueError("state_bits must be 8 or 32")
        self.params, self.grads, self.control = params, grads, control
        self.lr, self.betas, self.eps = lr, tuple(betas), eps
        self.weight_decays, self.lr_factors, self.bits, self.seed = decays, factors, bits, int(seed)
        self.t = 0

        numels = [p.numel() for p in params]
        room = {8: 0, 32: 0}
        self._at = []  # first element of each tensor in its state buffers
        for k, b in zip(numels, bits):
            self._at.append(room[b])
            room[b] += -(-k // L.STATE_BLOCK) * L.STATE_BLOCK
        if room[8] > MAX_POSITIONS:
            raise ValueError("more than 2^36 elements with 8-bit states in one list")
        wide, narrow = any(b == 32 for b in bits), any(b == 8 for b in bits)
        f32 = dict(dtype=torch.float32, device=device)
        self.exp_avg = torch.zeros(room[32], **f32) if wide else None
        self.exp_avg_sq = torch.zeros(room[32], **f32) if wide else None
        codes = torch.zeros(2, room[8], dtype=torch.uint8, device=device) if narrow else None
        self.codes_m = codes[0].view(torch.float8_e4m3fn) if narrow else None
        self.codes_r = codes[1].view(torch.float8_e4m3fn) if narrow else None
        self.scales = torch.zeros(room[8] // L.STATE_BLOCK, 2, **f32) if narrow else None

        first, chunk_tensor = _chunks(numels, L.PARAM_CHUNK)
        rows = []
        for i, (p, g, at) in enumerate(zip(params, grads, self._at)):
            if bits[i] == 32:
                m, v, s = self.exp_avg.data_ptr() + 4 * at, self.exp_avg_sq.data_ptr() + 4 * at, None
            else:
                m, v = self.codes_m.data_ptr() + at, self.codes_r.data_ptr() + at
                s = self.scales.data_ptr() + 8 * (at // L.STATE_BLOCK)
            rows.append(L.MuonParam(p.data_ptr(), g.data_ptr(), m, v, s, numels[i], at, first[i], decays[i], factors[i],
                                    dtype_code(p), dtype_code(g), bits[i], 0))
        tensors = _table((L.MuonParam * n)(*rows), device)
        chunks = torch.from_numpy(chunk_tensor).to(device)
        self.desc = L.MuonParamList(n, first[-1], tensors.data_ptr(), chunks.data_ptr())
        self.hyper, self._now = L.MuonAdamWHyper(0.0, 0.0, 0.0, 0.0, self.seed, 0), None
        self.elements = sum(numels)
        self._own(device, [self.exp_avg, self.exp_avg_sq, codes, self.scales, tensors, chunks,
                           None if control is None else control.block])

    def step(self, stream=None) -> None:
        now = (self.seed, self.lr, self.eps, *self.betas)
        if now != self._now:  # they may be set between steps
            h = self.hyper
            h.seed, h.lr, h.eps, h.beta1, h.beta2 = now
            self._now = now
        control, raw, here = self.control, self._on(stream), self._here()
        if control is None and self._capturing(stream, here):
            raise RuntimeError("capturing a step needs a control block: its replays would all use the same t")
        self._call(here, L.muon_adamw_multi, self.desc, self.hyper, self.t + 1, None if control is None else control.data_ptr(), raw)
        if control is None:
            self.t += 1

    def _state(self, i):
        """The state of tensor i as views: (m, v), or (codes, codes, scales)."""
        at, n = self._at[i], self.params[i].numel()
        if self.bits[i] == 32:
            return [self.exp_avg[at:at + n], self.exp_avg_sq[at:at + n]]
        b = L.STATE_BLOCK
        return [self.codes_m[at:at + n], self.codes_r[at:at + n], self.scales[at // b:at // b + -(-n // b)]]

    def moments(self, i):
        """(m, v) of tensor i as new fp32 tensors of its shape."""
        shape, st = self.params[i].shape, self._state(i)
        if self.bits[i] == 32:
            return st[0].clone().view(shape), st[1].clone().view(shape)
        s = st[2].repeat_interleave(L.STATE_BLOCK, 0)[:st[0].numel()]
        m, r = st[0].float() * s[:, 0], st[1].float() * s[:, 1]
        return m.view(shape), r.square().view(shape)

    def state_dict(self) -> dict:
        """The step count, every tensor's state (host copies: m and v, or the
        codes of m and r as uint8 and their scales) and the hyperparameters.  Of
        a control block it holds the step count; ``StepControl.state_dict()``
        has the rest."""
        def host(x):
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            return x.detach().to("cpu", copy=True)

        step = self.t if self.control is None else int(self.control.step.item())
        return {"step": step, "state": [[host(x) for x in self._state(i)] for i in range(len(self.params))],
                "bits": list(self.bits),
                "hyper": {"lr": self.lr, "betas": list(self.betas), "eps": self.eps, "seed": self.seed}}

    def check_state(self, state: dict) -> None:
        """Raises where load_state_dict() would refuse the state."""
        mine = [self._state(i) for i in range(len(self.params))]
        if list(state.get("bits", [])) != list(self.bits) or len(state["state"]) != len(mine) or any(
                len(a) != len(b) or any(x.shape != y.shape for x, y in zip(a, b)) for a, b in zip(state["state"], mine)):
            raise ValueError("the state was saved for differently shaped tensors or other state widths")

    def load_state_dict(self, state: dict) -> None:
        """Restores state_dict()'s state (weight decays and lr factors are the
        constructor's).  With a control block its step count is set too."""
        self.check_state(state)
        mine = [self._state(i) for i in range(len(self.params))]
        for i, (saved, own) in enumerate(zip(state["state"], mine)):
            for x, y in zip(saved, own):
                (y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y).copy_(x)
            # a block's maximum covers the codes behind the tensor too: none may stay from before
            end, n = self._at[i] + self.params[i].numel(), -self.params[i].numel() % L.STATE_BLOCK
            for buf in (self.exp_avg, self.exp_avg_sq) if self.bits[i] == 32 else (self.codes_m, self.codes_r):
                (buf.view(torch.uint8) if buf.dtype == torch.float8_e4m3fn else buf)[end:end + n].zero_()
        h = state["hyper"]
        self.lr, self.betas, self.eps = h["lr"], tuple(h["betas"]), h["eps"]
        self.seed = self.hyper.seed = int(h["seed"])
        if self.control is None:
            self.t = int(state["step"])
        else:
            self.control.step.fill_(int(state["step"]))
        _settle(self.device)
