"""The order of generation on a stream of the caller's, on the CPU with stand-ins for the streams: every
call of drafter, pool and target happens while that stream is the current one (so that torch's
operations between them are on it too), after it has waited for the caller's, which waits for it at the end."""
from contextlib import contextmanager
from types import SimpleNamespace

import pytest
import torch

from block_diffusion_drafter_kv_gb300.generate import spec_generate
from synthetic_target import TinyTarget, greedy_reference
from test_generate_logprobs_host import IDS, Scoring, target


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.device = name, log, torch.device("cpu")

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))


@pytest.fixture
def streams(monkeypatch):
    log = []
    caller, side = Stream("caller", log), Stream("side", log)
    current = [caller]

    @contextmanager
    def on(s):
        current.append(s)
        try:
            yield
        finally:
            current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    return log, current, side


def watched(obj, names, log, current):
    for n in names:
        def call(*a, _f=getattr(obj, n), _n=n, **kw):
            assert kw.get("stream") in (None, current[-1])
            log.append((current[-1].name, _n))
            return _f(*a, **kw)
        setattr(obj, n, call)
    return obj


def test_everything_runs_on_the_stream_between_two_waits(streams):
    log, current, side = streams
    d = watched(Scoring(1024, 8, 77), ("inject", "draft", "verify", "logprobs"), log, current)
    d.pages = watched(SimpleNamespace(reserve=lambda length, n, rows, batch, slots=None, stream=None: None,
                                      release=lambda length, batch, stream=None: None), ("reserve", "release"), log, current)
    t = watched(target(), ("prefill", "forward_block", "truncate"), log, current)
    out, st = spec_generate(d, t, IDS, 20, stream=side, logprobs=2)
    assert out == greedy_reference(target(), IDS, 20) and len(st.token_logprobs) == 20
    assert log[0] == ("side", "waits for", "caller") and log[-1] == ("caller", "waits for", "side")
    assert {e[0] for e in log[1:-1]} == {"side"}
    assert {e[1] for e in log[1:-1]} == {"inject", "draft", "verify", "logprobs", "reserve", "release", "prefill", "forward_block", "truncate"}
    assert current[-1].name == "caller"


def test_the_caller_waits_after_an_error_too(streams):
    log, current, side = streams

    class Broken(TinyTarget):
        def forward_block(self, tokens):
            raise ValueError("the target's own")

    with pytest.raises(ValueError):
        spec_generate(Scoring(1024, 8, 77), Broken(1024, 256, seed=3, bias_token=77, bias=4.8, device="cpu"), IDS, 20, stream=side)
    assert log == [("side", "waits for", "caller"), ("caller", "waits for", "side")] and current[-1].name == "caller"
