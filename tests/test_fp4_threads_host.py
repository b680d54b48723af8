"""A 4-bit layer's kept casts as its threads see them, without a GPU."""
import types

import pytest
import torch

from quantised_linear_layers_gb300 import fp4


class Stream:
    def __init__(self):
        self.waited = []

    def record_event(self):
        return object()

    def wait_event(self, event):
        self.waited.append(event)


class Buf:
    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


@pytest.mark.parametrize("in_between_wants_dgrad", [False, True])
def test_a_call_between_any_two_steps_of_another(monkeypatch, in_between_wants_dgrad):
    """After every attribute that one call sets, another call comes in on a stream of its own: it gets a cast with all
    that it asked for and has waited for the event behind that very cast, or made it itself."""
    now = [Stream()]
    made = {}                                            # cast -> (stream, its last event)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[0])
    calls = []

    class Layer(fp4.FP4Linear):
        armed = False

        def _cast(self, dgrad):
            buf = lambda: types.SimpleNamespace(buf=Buf())  # noqa: E731
            c = types.SimpleNamespace(dgrad=dgrad, w=buf(), wt=buf() if dgrad else None)
            made[id(c)] = (c, now[0])
            return c

        def __setattr__(self, name, value):
            super().__setattr__(name, value)
            if self.armed:
                object.__setattr__(self, "armed", False)
                mine, now[0] = now[0], Stream()
                calls.append((self.fp4_weight(in_between_wants_dgrad), now[0], in_between_wants_dgrad))
                now[0] = mine
                object.__setattr__(self, "armed", True)

    layer = Layer(8, 4)
    events = {}
    record = Stream.record_event

    def record_event(self):
        e = record(self)
        events[id(e)] = (e, self)
        return e

    monkeypatch.setattr(Stream, "record_event", record_event)
    object.__setattr__(layer, "armed", True)
    for _ in range(2):
        for dgrad in (False, True, False):
            now[0] = Stream()
            calls.append((layer.fp4_weight(dgrad), now[0], dgrad))
        with torch.no_grad():
            layer.weight.add_(1)                         # a new version: cast anew
    assert len(calls) > 6
    for cast, stream, dgrad in calls:
        assert cast.dgrad or not dgrad
        maker = made[id(cast)][1]
        if maker is not stream:
            assert any(events[id(e)][1] is maker for e in stream.waited)
            assert all(stream in c.buf.streams for c in (cast.w, cast.wt) if c is not None)
