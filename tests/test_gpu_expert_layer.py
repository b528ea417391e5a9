"""examples/expert_layer.py: the operators together, as a layer of experts uses them.

The bounds are what the number formats leave.  fp8: E4M3 values have a relative rounding error of
at most 2^-4, uniform in size over an octave, so 2^-4 / sqrt(3) * 3/4 = 0.027 rms; a random product
of two such operands is off by sqrt(2) times that, 0.038, and three products follow one another,
each again on rounded inputs: sqrt(3) * 0.038 = 0.066; twice that is allowed.  bf16: 2^-8 / sqrt(3)
* 3/4 = 0.0017 rms per rounding; the longest path (the gradient of h) has some fourteen roundings,
sqrt(14) * 0.0017 = 0.0063; twice that is allowed."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "expert_layer.py")


@pytest.mark.parametrize("rows,dim,hidden,experts", [(96, 512, 384, 8), (5, 264, 200, 16), (300, 384, 640, 3)])
def test_expert_layer(gemm_lib, cuda_device, rows, dim, hidden, experts):
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    served, errors = layer.main(rows, dim, hidden, experts)
    assert served <= 0.132
    assert all(v <= 0.0126 for v in errors.values()), errors
