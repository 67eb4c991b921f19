"""examples/expert_layer.py: the feed-forward operators and the all-reduce as a decode step runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# The activation is rounded to e4m3 once on the way, by up to 2^-4 of a value and 2^-4 / sqrt(3) = 0.036 in the root mean square; the
# bfloat16 roundings (gate and up, the down products, the weighted and the all-reduced sums, h: 2^-8 at most each, h's
# relative to the sum of a layer as to h, which is of the same size) add less than 0.012.
@pytest.mark.parametrize("args", [["--ranks", "1", "--layers", "2"], ["--ranks", "2"], ["--ranks", "4", "--tokens", "33", "--layers", "2", "--inner", "512"],
                                  ["--ranks", "2", "--tokens", "1", "--experts", "8", "--chosen", "8"]])
def test_expert_layers(example, args):
    worst, same = example.main(args)
    assert same
    assert worst < 0.05
