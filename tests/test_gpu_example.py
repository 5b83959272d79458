"""The example of three token mixers in one model runs and agrees with itself."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("lens,steps", [((37, 1, 200, 130), 5), ((5,), 2), ((300, 64, 129, 31, 1, 90), 1)])
def test_prompts_then_steps_are_longer_prompts(lens, steps):
    # each of three layers rounds to bf16 four times on its way (norm, projection, mixer, product), by
    # at most 2^-8 each and independently between the two runs: sqrt(2) * 12 * 2^-8
    assert load_example().check(lens, steps) <= 2 ** 0.5 * 12 * 2.0 ** -8
