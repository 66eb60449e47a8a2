"""The example layer (router, routed experts, shared expert on 4-bit weights)
against its own fp32 reference: bf16 outputs of two calls and their sum, three
roundings of 2^-9, and codes of h that fall to the other side of an edge (one in
10^4 or fewer, a few per cent of a term): within 2^-7 in the 2-norm."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp4_moe_layer.py")
    spec = importlib.util.spec_from_file_location("fp4_moe_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("tokens,experts,top_k,hidden,inner,groups", [
    (1, 64, 6, 1024, 512, 8), (32, 64, 6, 512, 288, 8), (300, 16, 2, 256, 160, 4), (700, 8, 2, 288, 96, 1)])
def test_layer(example, fmt, tokens, experts, top_k, hidden, inner, groups):
    assert example.run(tokens, experts, top_k, hidden, inner, fmt, groups, (groups + 1) // 2) <= 2.0 ** -7
