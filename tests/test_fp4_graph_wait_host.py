"""A captured forward uses casts that an earlier call made on whatever stream it
had: the host waits for them, since a capture cannot wait for an event from
outside. Without a GPU."""
import types

import pytest
import torch

from quantised_linear_layers_gb300 import fp4, ops


@pytest.mark.parametrize("same_stream", [False, True])
def test_the_event_behind_the_casts_is_waited_for(monkeypatch, same_stream):
    class Weight:
        is_cuda, device, dtype, requires_grad, _version = True, "cuda:0", torch.bfloat16, False, 0

        def data_ptr(self):
            return 64

        def detach(self):
            return self

    class Layer(fp4.FP4Linear):
        weight = Weight()

        def _cast(self, dgrad):
            return types.SimpleNamespace(dgrad=dgrad, w=None, wt=None)

    event = object()
    stream = [types.SimpleNamespace(record_event=lambda: event, wait_event=lambda e: None)]
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream[0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    held = []
    monkeypatch.setattr(ops, "_hold_in_graph", lambda *args: held.append(args))
    layer = fp4.FP4Linear(8, 4)
    layer.__class__ = Layer
    made = layer.fp4_weight(False)
    if not same_stream:
        stream[0] = types.SimpleNamespace()
    capturing[0] = True
    assert layer.fp4_weight(False) is made
    assert held == [(made, event)]
