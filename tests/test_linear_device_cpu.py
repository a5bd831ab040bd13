"""The linear-attention and norm calls launch on their tensors' device, current
or not. On the host: tensors that say they are on cuda:1, a library that notes
which device is current when it is called, and torch.cuda's current device as a
variable."""
import contextlib

import pytest
import torch

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import _linear


class OnDevice1(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 1)

    recorded = []  # (storage, stream) of the tensors that a stream was recorded for

    def get_device(self):
        return 1

    def record_stream(self, stream):
        OnDevice1.recorded.append((self.data_ptr(), stream))

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        kwargs.pop("device", None)
        return super().__torch_function__(func, types, args, kwargs)


def _on1(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)


class Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


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
    monkeypatch.setattr(torch.cuda, "stream", lambda s: device(s.device.index))
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw).as_subclass(OnDevice1))
    monkeypatch.setattr(_linear, "load", Library)
    monkeypatch.setattr(_linear, "_stream", lambda index: 0)
    _linear._size.cache_clear()
    _linear._weight_grad_bytes.cache_clear()
    yield seen
    _linear._size.cache_clear()
    _linear._weight_grad_bytes.cache_clear()
    assert now == [0]


def _calls():
    x, g, s = _on1(1, 4, 2, 128), _on1(1, 4, 2), _on1(1, 2, 128, 128)
    p, pg, cu = x[0], g[0], _on1(2, dtype=torch.int32)
    slots = _on1(4, dtype=torch.int32)
    pool = _on1(4, 2, 128, 128)
    return {
        "kda_linear_prefill": lambda **kw: kda.linear_prefill(x, x, x, g, s, **kw),
        "kda_linear_varlen_prefill": lambda **kw: kda.linear_varlen_prefill(p, p, p, pg, cu, s, **kw),
        "kda_linear_prefill_backward": lambda **kw: kda.linear_prefill_backward(x, x, x, g, x, s, **kw),
        "kda_linear_varlen_prefill_backward":
            lambda **kw: kda.linear_varlen_prefill_backward(p, p, p, pg, p, cu, s, **kw),
        "kda_linear_decode_step": lambda **kw: kda.linear_decode_step(p, p, p, pg, pool, **kw),
        "kda_linear_decode_step_slots": lambda **kw: kda.linear_decode_step_slots(p, p, p, pg, pool, slots, **kw),
        "kda_qk_norm_rope": lambda **kw: kda.qk_norm_rope(q=x, k=x, **kw),
        "kda_qk_norm_rope_backward": lambda **kw: kda.qk_norm_rope_backward(x, x, x, x, **kw),
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


@pytest.mark.parametrize("name", list(_calls()))
def test_inputs_of_a_call_on_a_stream_are_kept_for_it(launches, name, monkeypatch):
    """A tensor that is let go of after the call keeps its memory until the stream is past it."""
    stream, given = Stream(1), []
    entry = getattr(kda, name[4:])

    def note(*args, **kw):
        given.extend(t.data_ptr() for t in (*args, *kw.values()) if isinstance(t, torch.Tensor))
        return entry(*args, **kw)
    monkeypatch.setattr(kda, name[4:], note)
    OnDevice1.recorded.clear()
    _calls()[name]()
    assert given and not OnDevice1.recorded
    given.clear()
    _calls()[name](stream=stream)
    assert sorted(p for p, s in OnDevice1.recorded if s is stream) == sorted(given)
