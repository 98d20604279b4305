"""A workspace that a call allocates lies on its matrices' device (CPU: the
library's calls are stubs, the matrices have no memory)."""

import pytest
import torch

from matrix_aware_optimizer_step_amd import muon as mu


@pytest.mark.parametrize("device", [None, "cpu"])
def test_orthogonalize_grouped_takes_its_matrices_device(monkeypatch, device):
    asked = []

    def workspace(nbytes, where):
        asked.append(torch.device(where) if where is not None else None)
        return torch.empty(nbytes, dtype=torch.uint8)

    monkeypatch.setattr(mu, "workspace", workspace)
    monkeypatch.setattr(mu.L, "muon_orthogonalize_grouped_workspace", lambda *a: 256)
    monkeypatch.setattr(mu.L, "muon_orthogonalize_grouped", lambda *a: None)
    x = torch.empty(2, 8, 16, device="meta")
    mu.orthogonalize_grouped([x], [torch.empty_like(x)], device=device, stream=_Stream())
    assert asked == [torch.device(device or "meta")]


class _Stream:
    cuda_stream = 0
