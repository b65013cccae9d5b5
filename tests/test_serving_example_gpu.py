"""The serving example end to end: a prompt call and decode steps of a layer against plain attention (GPU).

The bound on max |error| / rms(output).  An output of the layer is a sum over ranks and heads of out-projected values, so
errors average: with u = 2^-8 the relative half step of bf16, the projections (u, once each for q, k, v), the rotated q
and k (u), the weights (u), the attention's output (u) and the layer's (u) add at most ~8 u to a term of the size of the
output, and the largest of the ~2e5 outputs is at most 6 rms: 6 * 8 * 2^-8 < 0.19 if every rounding went the same way.
An 8-bit cache rounds every key and value by up to 2^-4 (and once more when a page's scale grows): 6 * 2 * 2^-4 = 0.75
more if all went the same way."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from comm_gemm_tile_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_attention.py")
    spec = importlib.util.spec_from_file_location("serve_attention", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("cache,bound", [("bf16", 0.19), ("e4m3", 0.94)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_prompts_then_steps(example, cache, bound, window, sinks):
    error, _ = example.run(cache=cache, window=window, sinks=sinks)
    assert error <= bound, error
