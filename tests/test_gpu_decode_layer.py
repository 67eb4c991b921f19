"""examples/decode_layer.py: the operators and the all-reduce as a decode step runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# An e4m3 rounding is off by up to 2^-4 of a value and 2^-4 / sqrt(3) in the root mean square, 0.036; the bfloat16
# roundings on the way (projections, partial sums, the all-reduce: each 2^-8 at most) add less than 0.01.
@pytest.mark.parametrize("args", [["--ranks", "1", "--steps", "2"], ["--ranks", "2"],
                                  ["--ranks", "4", "--requests", "9", "--steps", "3", "--layers", "2"]])
def test_decode_layers(example, args):
    worst, same = example.main(args)
    assert same
    assert worst < 0.046
