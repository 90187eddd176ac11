"""The example that runs the microscaled 4-bit operators and the norm together:
its training has to learn, and a token alone has to agree with the batch."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_layer_example(fmt):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp4_layer.py")
    spec = importlib.util.spec_from_file_location("fp4_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, apart = example.main(["--rows", "640", "--width", "384", "--steps", "20", "--fmt", fmt])
    # two independent weight matrices of unit gain differ by a mean square of 2; a step at
    # rate 0.5 leaves 1 - 1 + 0.25 (1 + 384 / 640) = 0.4 of it, down to the noise of 4-bit
    # weights and activations (two relative errors of about 0.1 each: 0.02 to 0.03)
    assert losses[-1] < 0.1 * losses[0]
    # the same operands but for the bf16 rounding of the norm's output and its tensor
    # scale, which move some codes: no more than the quantization error itself
    assert apart < 0.1
