"""The README's Python lines: every call takes its arguments as the package's
function does, and the lines of one model agree on its scale, norm and state."""
import inspect
import os
import re
import sys
import types

import kda_gated_delta_chunkwise_gb300 as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Tensor:
    """Stands for any tensor, or a dict of them."""
    def __getitem__(self, key):
        return Tensor()


def _calls(monkeypatch):
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    section = text[text.index("## Use from Python"):]
    lines = re.findall(r"^    (.*)$", section[:section.index("\n`kda.")], flags=re.M)
    calls = {}
    fake = types.ModuleType("kda")

    def stand_in(name):
        real = getattr(kda, name)

        def call(*args, **kw):
            bound = inspect.signature(real).bind(*args, **{k: v for k, v in kw.items() if k != "stream"})
            bound.apply_defaults()
            calls[name] = bound.arguments
            return (Tensor(), Tensor()) if "prefill" in name and "backward" not in name or name == "qk_norm_rope" \
                else Tensor()
        return call
    for name in dir(kda):
        if callable(getattr(kda, name)) and not isinstance(getattr(kda, name), type):
            setattr(fake, name, stand_in(name))
    monkeypatch.setitem(sys.modules, "kda_gated_delta_chunkwise_gb300", fake)

    class Names(dict):
        def __missing__(self, name):
            self[name] = Tensor()
            return self[name]
    names = Names(torch=None)
    exec("\n".join(lines), names)
    return calls, names


def test_the_lines_of_one_model_agree(monkeypatch):
    calls, names = _calls(monkeypatch)
    forward, step, back = (calls[f"linear_{n}"] for n in ("prefill", "decode_step", "prefill_backward"))
    assert forward["scale"] == step["scale"] == back["scale"] != 1.0
    assert forward["decay"] == step["decay"] == back["decay"]
    assert back["initial_state"] is forward["initial_state"] is names["s0"]
    assert calls["qk_norm_rope"]["norm"] == calls["qk_norm_rope_backward"]["norm"]
    assert calls["prefill_backward"]["initial_state"] is calls["prefill"]["initial_state"]
