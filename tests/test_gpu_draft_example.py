"""The drafting example: it runs, and what it keeps are tokens of the vocabulary, as many as it counts."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "drafted_tree.py")


@pytest.mark.parametrize("steps", [1, 6])
def test_steps(cuda_dev, steps):
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("drafted_tree", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    texts, stood = example.run(steps)
    assert sum(len(t) for t in texts) == len(texts) * (steps + 1) + stood and 0 <= stood <= len(texts) * steps * example.LEVELS
    assert all(0 <= x < example.VOCAB for t in texts for x in t)
    assert texts == example.run(steps)[0]
