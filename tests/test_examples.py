"""The examples run, and what they compute holds together."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
def test_hybrid_layers():
    """Training lowers the loss, and generating token by token gives the logits
    of a pass over the whole text.  The two differ by the bf16 roundings along
    the path (about 16 stored activations, half a step of 2^-8 each)."""
    r = load("hybrid_layers").main(40)
    assert r["last"] < r["first"]
    assert r["difference"] <= 16 * 2 ** -8 * r["largest"], r
