"""CPU checks of the expert operators' host side: whose memory a call's results are."""

import torch

from matrix_aware_optimizer_step_amd import muon as mu


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
