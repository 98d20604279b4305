"""Workspaces that a call allocates for itself are memory of the stream it runs
on: a block of the current stream's may still be in use by kernels queued
there, which the call does not wait for."""

import pytest
import torch

from tests.test_gpu_expert_edges import owner

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_workspaces_are_memory_of_the_calls_stream(monkeypatch, handle):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    from matrix_aware_optimizer_step_amd import muon as mu
    from matrix_aware_optimizer_step_amd import soap
    made = []
    monkeypatch.setattr(mu, "workspace", lambda *a, f=mu.workspace: made.append(f(*a)) or made[-1])
    s = torch.cuda.Stream()
    stream = s.cuda_stream if handle else s
    g = torch.randn(2, 64, 96, device="cuda")
    mom, nout, out = torch.zeros_like(g), torch.empty_like(g), torch.empty_like(g)
    sums = torch.zeros(2, device="cuda")
    spd = torch.randn(2, 64, 64, device="cuda")
    q = torch.eye(64, device="cuda").repeat(2, 1, 1)
    torch.cuda.synchronize()
    mu.momentum(g, mom, nout, sums, stream=stream)
    mu.momentum_grouped([g], [mom], [nout], [sums], stream=stream)
    mu.orthogonalize(nout, out, sums, stream=stream)
    mu.orthogonalize_grouped([nout], [out], [sums], stream=stream)
    soap.qr(spd, q, stream=stream)
    torch.cuda.synchronize()
    assert len(made) == 5 and {owner(t) for t in made} == {s.cuda_stream}
    assert out.isfinite().all() and q.isfinite().all()
