"""The example layer: prompts, then single tokens from a captured graph."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")


@pytest.mark.parametrize("steps", [1, 40])
def test_layer(cuda_dev, steps):
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("attention_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    prompt, last, _ = example.run(steps)
    assert 0.0 < prompt <= 1.0 and 0.0 < last <= 1.0
