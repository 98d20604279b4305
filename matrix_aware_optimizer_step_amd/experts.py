"""Mixture-of-experts operators of libmuon355 for torch: the routing of tokens
to experts with its gradient and the step of the bias that balances it, and the
tokens' sums over their experts.

Together with the block codes (``blocks``) they run the layers whose expert
matrices the optimizer step updates::

    r = route(logits, 8, bias=balance.bias, loads=balance.loads, align=128)
    a, at = quantize(x, pairs=(r.pairs, 8), order="both")  # rows by expert
    y = expert_matmul(a, codes.codes, r.offsets)
    out = expert_sum(y, r.slots, r.weights)

and backward, from the gradient of ``out``::

    g, gt = quantize(grad, pairs=r.pairs, weights=r.weights, order="both")
    expert_grad(gt, at, r.offsets, out=weight_grads, accumulate=True)
    grad_x = expert_sum(expert_matmul(g, codes.transposed, r.offsets), r.slots)
    grad_logits = route_backward(logits, r, expert_dot(grad, y, r.slots))

Every call only enqueues kernels, on the current stream of its tensors' device
or on ``stream``; there is no CPU path.
"""

from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from . import _lib as L
from .blocks import _enqueue, _filled, _matrix, _need, _same_device
from .muon import _made_on, dtype_code
from .multi import StepControl, _OnDevice, _settle

NO_EXPERT = -1
_MOST = torch.finfo(torch.float32).max


@dataclass
class Routing:
    """What ``route`` found.

    ``experts`` int32 [tokens, k]: the chosen ones, best first, -1 for none.
    ``weights`` float32 [tokens, k].  ``slots`` int32 [tokens, k]: each pair's row in
    the order by expert, or -1.  ``pairs`` int32 [rows]: each row's pair (token * k + j),
    or -1.  ``offsets`` int32 [experts + 1]: each expert's first row.  The last
    three are None with ``order=False``.
    """
    experts: torch.Tensor
    weights: torch.Tensor
    slots: torch.Tensor | None
    pairs: torch.Tensor | None
    offsets: torch.Tensor | None
    score: str
    renormalize: bool
    scale: float

    @property
    def k(self) -> int:
        return self.experts.shape[1]


def _check_logits(logits) -> None:
    _need(logits.dim() == 2, "logits must be [tokens, experts]")
    _need(logits.stride(1) == 1 or logits.shape[1] <= 1, "logits must be row-major (last stride 1)")
    if not 1 <= logits.shape[1] <= L.MAX_EXPERTS:
        raise ValueError(f"experts outside [1, {L.MAX_EXPERTS}]")


def _ld(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _check(t, shape, dtype, what, device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")


@functools.lru_cache(maxsize=256)
def _sizes(tokens, experts, k, align, order):
    """Rows of the order, and 32-bit words of the workspace."""
    rows = L.muon_route_capacity(tokens, experts, k, align) if order else 0
    _need(rows > 0 or not order, "align outside [1, 65536], or an order of more than 2^22 tokens or 2^31-1 rows")
    return rows, -(-L.muon_route_workspace(tokens, experts) // 4)


def route(logits: torch.Tensor, k: int, *, bias: torch.Tensor | None = None, score: str = "softmax", groups: int = 1,
          top_groups: int = 1, group_best: int = 2, renormalize: bool = True, scale: float = 1.0,
          mask: torch.Tensor | None = None, align: int = 1, loads: torch.Tensor | None = None, order: bool = True,
          stream=None) -> Routing:
    """Tokens to their k best experts (``muon_route``; muon355.h has the definition).

    ``logits``: bfloat16 or float32 [tokens, experts], a row stride of its own.
    ``bias`` (float32 [experts]) is added to the scores that choose, not to the
    weights.  ``groups`` runs of experts are marked by the sum of their ``group_best``
    (1 or 2) best, and the ``top_groups`` best stay.  ``mask`` (bool [tokens]): False
    sends a token nowhere (padding).  A logit of -inf takes its expert out.
    ``align``: each expert's rows are rounded up to a multiple of it (128 where
    ``expert_grad`` follows, so that no two experts share a block).  ``loads``
    (int32 [experts]): each expert's tokens are added to it.  ``order=False``
    leaves the order by expert out.
    """
    _check_logits(logits)
    tokens, experts = logits.shape
    device = logits.device
    if score not in L.SCORES:
        raise ValueError(f"score must be one of {sorted(L.SCORES)}")
    if not 1 <= k <= min(L.MAX_CHOSEN, experts):
        raise ValueError(f"k outside [1, min({L.MAX_CHOSEN}, experts)]")
    if bias is not None:
        _check(bias, (experts,), torch.float32, "bias", device)
    if mask is not None:
        _check(mask, (tokens,), torch.bool, "mask", device)
    if loads is not None:
        _check(loads, (experts,), torch.int32, "loads", device)
    rows, ws = _sizes(max(tokens, 1), experts, k, align, order)
    if tokens == 0:
        rows = -(-experts * (align - 1) // align) * align if order else 0
    # one buffer: experts, slots, pairs, offsets, and a workspace on a multiple of 16 bytes
    n = tokens * k
    end = -(-(2 * n + rows + experts + 1) // 4) * 4 if order else -(-n // 4) * 4
    ints, weights = _made_on(stream, device, lambda: (
        torch.empty(end + ws, dtype=torch.int32, device=device),
        torch.empty((tokens, k), dtype=torch.float32, device=device)))
    found = Routing(ints.as_strided((tokens, k), (k, 1)), weights,
                    ints.as_strided((tokens, k), (k, 1), n) if order else None,
                    ints.as_strided((rows,), (1,), 2 * n) if order else None,
                    ints.as_strided((experts + 1,), (1,), 2 * n + rows) if order else None,
                    score, bool(renormalize), float(scale))
    if tokens == 0:
        if device.type != "cuda":
            raise RuntimeError("the tensors are not on a GPU (there is no CPU path)")
        if order:
            _filled(found.pairs, NO_EXPERT, stream)
            _filled(found.offsets, 0, stream)
        return found
    desc = L.MuonRoute(logits.data_ptr(), _ld(logits), tokens, experts, k, dtype_code(logits), L.SCORES[score],
                       1 if renormalize else 0, groups, top_groups, group_best, align, scale)
    at = ints.data_ptr()
    _enqueue(device, stream, (ints, weights), L.muon_route, desc, None if bias is None else bias.data_ptr(),
             None if mask is None else mask.data_ptr(), at, weights.data_ptr(), at + 4 * n if order else None,
             at + 8 * n if order else None, at + 8 * n + 4 * rows if order else None,
             None if loads is None else loads.data_ptr(), at + 4 * end, 4 * ws)
    return found


def route_backward(logits: torch.Tensor, routing: Routing, grad_weights: torch.Tensor, *,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of the logits that ``route`` was given, from the gradient of its
    weights (float32 [tokens, k]), in the logits' type."""
    _check_logits(logits)
    device = logits.device
    shape = (logits.shape[0], routing.k)
    _check(routing.experts, shape, torch.int32, "routing.experts", device)
    _check(routing.weights, shape, torch.float32, "routing.weights", device)
    _check(grad_weights, shape, torch.float32, "grad_weights", device)
    made = out is None
    if made:
        out = _made_on(stream, device, lambda: torch.empty(logits.shape, dtype=logits.dtype, device=device))
    else:
        _need(out.shape == logits.shape and out.dtype == logits.dtype and (out.stride(1) == 1 or out.shape[1] <= 1),
              "out must have the logits' shape and type and last stride 1")
        _same_device(device, out, "out")
    if logits.shape[0] == 0:
        return out
    desc = L.MuonRoute(logits.data_ptr(), _ld(logits), logits.shape[0], logits.shape[1], routing.k, dtype_code(logits),
                       L.SCORES[routing.score], int(routing.renormalize), 1, 1, 1, 1, routing.scale)
    _enqueue(device, stream, (out,) if made else (), L.muon_route_backward, desc, routing.experts.data_ptr(),
             routing.weights.data_ptr(), grad_weights.data_ptr(), out.data_ptr(), _ld(out))
    return out


def _check_slots(slots, device) -> None:
    if slots.dim() != 2 or not 1 <= slots.shape[1] <= L.MAX_CHOSEN:
        raise ValueError(f"slots must be [tokens, 1 .. {L.MAX_CHOSEN}]")
    _check(slots, slots.shape, torch.int32, "slots", device)


def expert_sum(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, *,
               out: torch.Tensor | None = None, dtype=None, stream=None) -> torch.Tensor:
    """Each token's sum of weights[t, j] * y[slots[t, j]] (weights None: ones),
    in fp32, rounded once to ``dtype`` (None: y's).  A slot of -1 adds nothing
    (a NaN weight is passed on).  ``out`` must not overlap y."""
    desc, device = _matrix(y, "y"), y.device
    _check_slots(slots, device)
    tokens, k = slots.shape
    if weights is not None:
        _check(weights, (tokens, k), torch.float32, "weights", device)
    shape, made = (tokens, y.shape[1]), out is None
    if made:
        out = _made_on(stream, device, lambda: torch.empty(shape, dtype=dtype or y.dtype, device=device))
    elif tuple(out.shape) != shape:
        raise ValueError(f"out must be {shape}, not {tuple(out.shape)}")
    _same_device(device, out, "out")
    od = _matrix(out, "out")
    if tokens == 0 or shape[1] == 0:
        return out
    if y.shape[0] == 0:
        return _filled(out, 0, stream)
    _enqueue(device, stream, (out,) if made else (), L.muon_expert_sum, desc, slots.data_ptr(),
             None if weights is None else weights.data_ptr(), k, od)
    return out


def expert_dot(grad: torch.Tensor, y: torch.Tensor, slots: torch.Tensor, *, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """The gradient of ``expert_sum``'s weights: <grad[t], y[slots[t, j]]>, float32 [tokens, k]."""
    gd, yd, device = _matrix(grad, "grad"), _matrix(y, "y"), y.device
    _check_slots(slots, device)
    tokens, k = slots.shape
    if tuple(grad.shape) != (tokens, y.shape[1]):
        raise ValueError(f"grad must be {(tokens, y.shape[1])}, not {tuple(grad.shape)}")
    _same_device(device, grad, "grad")
    made = out is None
    if made:
        out = _made_on(stream, device, lambda: torch.empty((tokens, k), dtype=torch.float32, device=device))
    else:
        _check(out, (tokens, k), torch.float32, "out", device)
    if out.numel() == 0:
        return out
    if y.numel() == 0:
        return _filled(out, 0, stream)
    _enqueue(device, stream, (out,) if made else (), L.muon_expert_dot, gd, yd, slots.data_ptr(), k, out.data_ptr())
    return out


def _rate(x) -> float:
    x = float(x)
    if not 0.0 <= x <= _MOST:  # (the library takes a float)
        raise ValueError("rate must be finite and >= 0")
    return x


class BalanceBias(_OnDevice):
    """The bias that keeps a router's experts evenly loaded, and the loads it
    goes by.

    Give ``bias`` and ``loads`` to ``route`` in every forward pass of a step; ``step()``
    (``OptimizerStep(balance=[...])`` calls it after its updates) moves each
    expert's bias by ``rate`` towards the mean load and starts the loads again from
    zero (``muon_balance_update``).  With a ``StepControl`` a skipped step leaves the bias as it is.
    With several GPUs sum ``loads`` over them first, with an all-reduce.
    """

    def __init__(self, experts: int, rate: float = 1e-3, device="cuda"):
        if not 1 <= experts <= L.MAX_EXPERTS:
            raise ValueError(f"experts outside [1, {L.MAX_EXPERTS}]")
        self.rate = _rate(rate)
        self.bias = torch.zeros(experts, dtype=torch.float32, device=device)
        self.loads = torch.zeros(experts, dtype=torch.int32, device=device)
        self._control = None  # the one of the last step
        self._own(self.bias.device, [self.bias, self.loads])

    def step(self, control: StepControl | None = None, stream=None) -> None:
        if control is not None and control.device != self.device:
            raise ValueError("control is on another device than the bias")
        if control is not None and control is not self._control:
            self._control = control
            self._buffers = [self.bias, self.loads, control.block]
            self._seen.clear()
        raw = self._on(stream)
        self._call(self._here(), L.muon_balance_update, self.bias.data_ptr(), self.loads.data_ptr(), self.bias.numel(),
                   self.rate, None if control is None else control.data_ptr(), raw)

    def state_dict(self) -> dict:
        return {"bias": self.bias.to("cpu", copy=True), "loads": self.loads.to("cpu", copy=True), "rate": self.rate}

    def check_state(self, state: dict) -> None:
        """Raises where load_state_dict() would refuse the state."""
        for key, own in (("bias", self.bias), ("loads", self.loads)):
            if key not in state or state[key].shape != own.shape:
                raise ValueError("the state was saved for another number of experts")
        if "rate" not in state:
            raise ValueError("the state was saved for something else than a balance bias")
        _rate(state["rate"])

    def load_state_dict(self, state: dict) -> None:
        self.check_state(state)
        self.bias.copy_(state["bias"])
        self.loads.copy_(state["loads"])
        self.rate = _rate(state["rate"])
        _settle(self.bias.device)
