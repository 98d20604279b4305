"""libmuon355: the Muon optimizer step on AMD Instinct MI355X (gfx950).

Momentum, Newton-Schulz orthogonalization and the shape-scaled update run in
hand-written HIP kernels behind the C ABI of include/muon355.h, and so does
the AdamW step for the parameters Muon does not take, and the gradient norm
that clips both.  Around the step stand the operators of the layers whose
matrices it updates: 8-bit block codes and their products, the routing of
tokens to experts and the experts' sums.  ``_lib`` is the ctypes binding (same
names as the C entry points); ``muon`` and ``multi`` turn torch tensors into
descriptors and hold the buffers of a whole step, ``blocks`` and ``experts`` do
so for the layers' operators.
"""

from . import _lib
from ._lib import (MUON_BF16, MUON_F32, MUON_SCALE_MATCH_RMS, MUON_SCALE_NONE, MUON_SCALE_ORIGINAL, MuonBatch,
                   MuonError)
from .blocks import BlockCodes, WeightCodes, block_matmul, expert_grad, expert_matmul, quantize
from .experts import BalanceBias, Routing, expert_dot, expert_sum, route, route_backward
from .multi import AdamWMulti, GradClip, StepControl
from .muon import (EPS, QUINTIC, AdamW, Batch, MuonStep, OptimizerStep, apply, apply_grouped, batch, is_muon_param,
                   momentum, momentum_grouped, orthogonalize, orthogonalize_grouped, workspace)

__all__ = ["_lib", "MUON_BF16", "MUON_F32", "MUON_SCALE_MATCH_RMS", "MUON_SCALE_NONE", "MUON_SCALE_ORIGINAL",
           "MuonBatch", "MuonError", "EPS", "QUINTIC", "Batch", "MuonStep", "apply", "apply_grouped", "batch",
           "momentum", "momentum_grouped", "orthogonalize", "orthogonalize_grouped", "workspace", "AdamW",
           "OptimizerStep", "is_muon_param", "AdamWMulti", "GradClip", "StepControl",
           "BlockCodes", "WeightCodes", "block_matmul", "expert_grad", "expert_matmul", "quantize",
           "BalanceBias", "Routing", "expert_dot", "expert_sum", "route", "route_backward"]
