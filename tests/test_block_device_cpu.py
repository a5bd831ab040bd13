"""The window attention, block norm and axes calls launch on their tensors'
device, current or not, and on a given stream of it alone; on the host, as
test_linear_device_cpu.py does it for the calls that were there before."""
import pytest
import torch

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import _block, _linear, _window
from test_linear_device_cpu import OnDevice1, Stream, _on1, launches  # noqa: F401 (a fixture)


@pytest.fixture
def seen(launches, monkeypatch):  # noqa: F811
    caches = [f for m in (_block, _window) for f in vars(m).values() if hasattr(f, "cache_clear")]
    for module in (_block, _window):
        monkeypatch.setattr(module, "load", _linear.load)
        monkeypatch.setattr(module, "_stream", _linear._stream)
    for f in caches:
        f.cache_clear()
    yield launches
    for f in caches:
        f.cache_clear()


def _calls():
    x, lse, w = _on1(1, 4, 2, 128), _on1(1, 4, 2), _on1(128)
    p, cu = x[0], _on1(2, dtype=torch.int32)
    cache, slots = _on1(4, 8, 2, 128), _on1(4, dtype=torch.int32)
    row, table, pos = _on1(4, 128), _on1(10, 8), _on1(2, 1, 4, dtype=torch.int32)
    win = dict(window=4, sinks=2)
    return {
        "kda_qk_norm_rope_axes": lambda **kw: kda.qk_norm_rope_axes(x, x, pos, table, (0, 0, 1, 1), **kw),
        "kda_qk_norm_rope_axes_backward":
            lambda **kw: kda.qk_norm_rope_axes_backward(x, x, x, x, pos, table, (0, 0, 1, 1), w, **kw),
        "kda_gated_norm": lambda **kw: kda.gated_norm(x=x, gate=x, **kw),
        "kda_gated_norm_backward": lambda **kw: kda.gated_norm_backward(x, x, x, w, **kw),
        "kda_residual_norm": lambda **kw: kda.residual_norm(residual=row, branch=row, **kw),
        "kda_residual_norm_backward": lambda **kw: kda.residual_norm_backward(row, row, row, row, w, **kw),
        "kda_window_attention": lambda **kw: kda.window_attention(x, x, x, **win, **kw),
        "kda_window_varlen_attention": lambda **kw: kda.window_varlen_attention(p, p, p, cu, **win, **kw),
        "kda_window_attention_backward": lambda **kw: kda.window_attention_backward(x, x, x, x, lse, x, **win, **kw),
        "kda_window_varlen_attention_backward":
            lambda **kw: kda.window_varlen_attention_backward(p, p, p, p, lse[0], p, cu, **win, **kw),
        "kda_window_cache_write": lambda **kw: kda.window_cache_write(p, p, cu, cache, cache, slots[:1], sinks=2, **kw),
        "kda_window_decode_step": lambda **kw: kda.window_decode_step(p, p, p, cache, cache, slots, slots, sinks=2, **kw),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_a_call_runs_on_its_tensors_device(seen, name):
    _calls()[name]()
    assert seen == [(name, 1)]


@pytest.mark.parametrize("name", list(_calls()))
def test_a_stream_of_another_device_is_refused(seen, name):
    _calls()[name](stream=Stream(1))
    assert seen == [(name, 1)]
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        _calls()[name](stream=Stream(0))
    assert len(seen) == 1


@pytest.mark.parametrize("name", list(_calls()))
def test_inputs_of_a_call_on_a_stream_are_kept_for_it(seen, name, monkeypatch):
    stream, given = Stream(1), []
    entry = getattr(kda, name[4:])

    def note(*args, **kw):
        given.extend(t.data_ptr() for t in (*args, *kw.values()) if isinstance(t, torch.Tensor))
        return entry(*args, **kw)
    monkeypatch.setattr(kda, name[4:], note)
    OnDevice1.recorded.clear()
    _calls()[name](stream=stream)
    assert given and sorted(p for p, s in OnDevice1.recorded if s is stream) == sorted(given)
