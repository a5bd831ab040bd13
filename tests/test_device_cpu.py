"""The delta-rule calls launch on their tensors' device, current or not (see
test_linear_device_cpu, whose tensors and streams these are)."""
import contextlib

import pytest
import torch

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import _binding
from test_linear_device_cpu import OnDevice1, Stream, _on1


@pytest.fixture
def launches(monkeypatch):
    """The devices that were current when the library was called."""
    now, seen = [0], []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        try:
            yield
        finally:
            now[0] = before

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace_bytes"):
                return lambda *a: 256
            return lambda *a: seen.append((name, now[0])) or 0

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw).as_subclass(OnDevice1))
    monkeypatch.setattr(_binding, "load", Library)
    monkeypatch.setattr(_binding, "_stream", lambda stream: None)
    yield seen
    assert now == [0]


def _calls():
    x, b, s = _on1(1, 4, 2, 128), _on1(1, 4, 2), _on1(1, 2, 128, 128)
    p, pb, cu, pool = x[0], b[0], _on1(2, dtype=torch.int32), _on1(4, 2, 128, 128)
    slot, slots = _on1(1, dtype=torch.int32), _on1(4, dtype=torch.int32)
    u, sc = _on1(1, 4, 2, 128, dtype=torch.uint8), _on1(1, 4, 2, 4, dtype=torch.uint8)
    return {
        "kda_prefill_gate": lambda **kw: kda.prefill(x, x, x, x, b, s, **kw),
        "kda_prefill_segmented": lambda **kw: kda.prefill_segmented(x, x, x, x, b, **kw),
        "kda_prefill_fp8": lambda **kw: kda.prefill_fp8(u, u, u, sc, sc, sc, x, b, **kw),
        "kda_varlen_prefill": lambda **kw: kda.varlen_prefill(p, p, p, p, pb, cu, **kw),
        "kda_varlen_prefill_slots": lambda **kw: kda.varlen_prefill_slots(p, p, p, p, pb, cu, pool, slot, **kw),
        "kda_decode_step": lambda **kw: kda.decode_step(q=p, k=p, v=p, alpha=p, beta=pb, state=pool, **kw),
        "kda_decode_step_slots": lambda **kw: kda.decode_step_slots(p, p, p, p, pb, pool, slots, **kw),
        "kda_prefill_backward_gate": lambda **kw: kda.prefill_backward(x, x, x, x, b, x, **kw),
        "kda_varlen_prefill_backward": lambda **kw: kda.varlen_prefill_backward(p, p, p, p, pb, p, cu, **kw),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_a_call_runs_on_its_tensors_device(launches, name):
    _calls()[name]()
    assert launches == [(name, 1)]


@pytest.mark.parametrize("name", list(_calls()))
def test_a_stream_of_another_device_is_refused(launches, name):
    _calls()[name](stream=Stream(1))
    assert launches == [(name, 1)]
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        _calls()[name](stream=Stream(0))
    assert len(launches) == 1
