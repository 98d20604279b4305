"""CPU checks of the expert operators' host side: whose memory a call's results
are, what the calls accept."""

import pytest
import torch

import matrix_aware_optimizer_step_amd as mx
from matrix_aware_optimizer_step_amd import _lib as L
from matrix_aware_optimizer_step_amd import muon as mu
from tests import test_experts_binding as B


class Within:
    """A context that notes what is entered."""

    def __init__(self, entered, what):
        self.entered, self.what = entered, what

    def __enter__(self):
        self.entered.append(self.what)

    def __exit__(self, *_):
        self.entered.remove(self.what)


def test_memory_is_made_within_the_calls_stream(monkeypatch):
    entered = []
    monkeypatch.setattr(torch.cuda, "device", lambda d: Within(entered, ("device", d)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: Within(entered, ("stream", s)))

    class Stream:
        cuda_stream = 1234

    s, device = Stream(), torch.device("cuda", 0)
    assert mu._made_on(s, device, lambda: list(entered)) == [("device", device), ("stream", s)] and not entered
    assert mu._made_on(None, device, lambda: list(entered)) == []              # the current stream
    assert mu._made_on(s, torch.device("cpu"), lambda: list(entered)) == []


def test_pairs_of_a_matrix_without_rows():
    """An empty batch's order still has rows of -1: quantize passes them on, and the library takes x without rows there
    only."""
    def refused(x, pairs, **kw):
        with pytest.raises(L.MuonError) as e:
            L.muon_block_quantize(x, pairs, None, 1, B.codes(rows=7, cols=200, **kw), None, 0)
        return e.value.status, str(e.value)

    # (nothing here reaches a launch: the codes are refused after x has been accepted)
    status, text = refused(B.dense(0, 200, base=None), B.FAKE, reserved=1)
    assert status == B.INVALID and "q: reserved" in text
    assert "x: 0 x 200" in refused(B.dense(0, 200, base=None), None)[1]
    assert "x: ld" in refused(B.dense(0, 200, base=None, ld=100), B.FAKE)[1]
    assert "codes' shape" in refused(B.dense(0, 199, base=None), B.FAKE)[1]


def test_a_workspace_is_enough_for_fewer_tokens():
    for experts in (1, 64, 100, 128, 512):
        sizes = [L.muon_route_workspace(t, experts) for t in (1, 63, 64, 65, 1000, 16383, 16384, 16385, 20000, 65535, 65536,
                                                                65537, 1 << 20)]
        assert sizes == sorted(sizes)
    assert L.muon_route_workspace(16385, 128) == L.muon_route_workspace(16384, 128) == 1024 * 128
    assert L.muon_route_workspace(16385, 127) <= L.muon_route_workspace(16385, 129)
    need = L.muon_route_workspace(16385, 128)
    with pytest.raises(L.MuonError) as e:
        L.muon_route(B.route_desc(tokens=16385, experts=128, ld=128), None, None, B.FAKE, B.FAKE, None, None, None, None,
                     B.FAKE, need - 1, 0)
    assert e.value.status == B.WORKSPACE


def test_a_rate_is_checked_before_a_step_begins():
    """The library refuses such a rate too, but only once the step's other updates are on their way."""
    for bad in (-0.1, float("nan"), float("inf"), 1e39):
        with pytest.raises(ValueError, match="rate"):
            mx.BalanceBias(4, bad, "cpu")
    own, other = mx.BalanceBias(4, 0.5, "cpu"), mx.BalanceBias(4, 0.25, "cpu")
    other.bias.fill_(1.0)
    for change in (lambda s: s.pop("rate"), lambda s: s.update(rate=-1.0), lambda s: s.update(rate=float("nan"))):
        state = other.state_dict()
        change(state)
        with pytest.raises(ValueError):
            own.check_state(state)
        with pytest.raises(ValueError):
            own.load_state_dict(state)
        assert not own.bias.any() and own.rate == 0.5  # nothing was loaded
    own.load_state_dict(other.state_dict())
    assert (own.bias == 1).all() and own.rate == 0.25
