"""The example of a served layer (examples/decode_layer.py): prompts and decoding steps through the packed
products, the cache and the attention together.  Against float32 arithmetic on the cache's contents the
attention may differ by its rounding to bfloat16 (2^-8 of the output) and by that of its probabilities to
float16 and the float32 sums of both sides (2^-11 + 2^-12 of sum_j w_j |v_j|, taken as at most 16 times the
largest output)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompts,steps", [((37, 5, 64, 1), 8), ((1,), 1), ((15, 16, 17), 2), ((130, 2), 31)])
def test_decode_layer(prompts, steps):
    assert load().run(prompts, steps) <= 2.0 ** -8 + 16 * (2.0 ** -11 + 2.0 ** -12)
