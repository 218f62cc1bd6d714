"""The steps' ``capture`` and the work that the caller has queued before it.  The order of the
calls is checked without a GPU, the results on one."""

import contextlib

import pytest
import torch

from test_q8_step import _prepare, _state
from tree_speculative_decoding_tsd_gb300.step import Q8TreeVerifyStep, TreeVerifyStep

gpu = pytest.mark.gpu


class FakeStream:
    """Records what is asked of it, in order."""

    def __init__(self, log, name):
        self.log, self.name, self.device = log, name, "cuda:0"

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))

    def synchronize(self):
        self.log.append((self.name, "synchronized"))


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("cls,method", [(TreeVerifyStep, "_round"), (Q8TreeVerifyStep, "run")])
def test_capture_follows_the_callers_stream(monkeypatch, cls, method, given):
    """The round before the recording waits for the stream that is current at the call."""
    log = []
    callers, other = FakeStream(log, "the caller's"), FakeStream(log, "the capture's")
    monkeypatch.setattr(torch.cuda, "Stream", lambda *a, **k: other)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: callers)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "CUDAGraph", lambda: "graph")
    monkeypatch.setattr(torch.cuda, "graph", lambda *a, **k: contextlib.nullcontext())
    monkeypatch.setattr(cls, method, lambda self, *a, **k: log.append(("round",)))
    step = object.__new__(cls)
    probs = torch.empty(1)
    args = (probs,) + (None,) * (8 if cls is TreeVerifyStep else 7)
    assert step.capture(*args, stream=other if given else None) == "graph"
    assert log == [("the capture's", "waits for", "the caller's"), ("round",),
                   ("the capture's", "synchronized"), ("round",)]


@gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("kind", ["gqa", "latent"])
def test_capture_behind_queued_rounds(kind, given):
    """A prompt and a round queued behind 50 ms of other work, and a capture without waiting
    for them: the state after its own round is that of the calls one after the other."""
    keep = 150

    def state_of(capture):
        s, step, cache, weights, probs, root, logits = _prepare(kind, 0, keep)
        args = (probs, root, s.q, cache, s.plen, s.kt, s.vt, logits, weights)
        stream = torch.cuda.Stream() if given else None
        more = s.normal(2, 3, s.Hkv, s.dk), None if s.latent else s.normal(2, 3, s.Hkv, s.dv)
        n = torch.tensor([3, 2], dtype=torch.int32, device=s.plen.device)
        torch.cuda.synchronize()
        if capture:
            torch.cuda._sleep(100_000_000)
        step.append(*more, n, cache, s.plen)
        step.run(*args)
        if capture:
            step.capture(*args, stream=stream)
        else:
            torch.cuda.synchronize()
            step.run(*args)
        torch.cuda.synchronize()
        assert int(step.err[0]) == 0
        return [step.out, step.lse] + _state(cache, weights, s.plen)

    want, got = state_of(False), state_of(True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
