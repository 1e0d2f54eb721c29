"""The example's layer runs, and its output and gradients are those of the plain layer but for 8-bit
roundings: at most 2^-4 of a value, evenly spread 2^-4 / sqrt(3) = 3.6 percent rms of the values that a
sum adds up.  Two roundings reach the output (the norm's rows and SwiGLU's), two more the gradient of
x (both products' rows on the way back), where half of each sum is the residual's, which is exact:
5.1 and 7.2 percent, twice that allowed."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,E,k,dff", [(300, 256, 8, 2, 256), (64, 384, 5, 3, 128)])
def test_example(T, d, E, k, dff):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "fp8_block_experts.py")
    spec = importlib.util.spec_from_file_location("fp8_block_experts", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out, dx, dweight = ex.run(T, d, E, k, dff)
    assert out < 0.102
    assert dx < 0.144
    assert dweight < 0.144
