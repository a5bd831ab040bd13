"""The example layer: decoding token by token against one prefill, and a
training step against what its gradient promises.

Tolerances. Outputs are bf16 (2^-9 relative) at four places one after the other
(q and k, o, y), and the prefill's P and state are rounded to bf16 too: 1e-2 of
the 2-norm is above 5 x 2^-9 with correlated errors. A step of 0.5 % of each
weight's norm against the gradient changes the loss by the first-order term and
a second-order one of the order of the step times the first; with bf16 outputs
the measured change of the loss carries their rounding as well: 20 %.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(kda):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "linear_attention_layer.py")
    spec = importlib.util.spec_from_file_location("linear_attention_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T,new", [(300, 5), (1, 2), (128, 1)])
def test_decode_follows_prefill(example, T, new):
    assert example.serve(example.Layer(), T=T, new=new) < 1e-2


def test_step_does_what_its_gradient_promises(example):
    before, promised, change = example.train(example.Layer(), rate=0.005)
    assert promised < 0 and change < 0
    assert abs(change - promised) < 0.2 * abs(promised)
