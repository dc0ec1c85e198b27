"""Layer norm on the GPU at the ends of its range: rows and gradients of far
apart scales."""
import numpy as np
import pytest

from test_gpu_layernorm import _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [128, 1032, 2048, 5120])
@pytest.mark.parametrize("xs,ds", [(1e16, 1e-12), (1e14, 1e-15), (1e-12, 1e12)])
def test_scales_far_apart(cuda_lib, width, dtype, xs, ds):
    # dx scales with ds / xs, within the format's range; nothing on the way may
    # leave fp32's (a product of two rstd would)
    rng = np.random.default_rng(width)
    x, dy, w, b = _case(rng, 37, width, dtype)
    _check(cuda_lib, x * xs, dy * ds, w, b, eps=0.0)
