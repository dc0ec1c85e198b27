"""Layer norm on the GPU at the ends of its range: constant rows, rows and
gradients of far apart scales."""
import numpy as np
import pytest
import torch

from ends_util import TORCH, draw
from test_gpu_layernorm import _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("width", [24, 40, 776, 1032, 2048, 5120, 10240])
def test_constant_rows_are_the_bias(cuda_lib, width, dtype):
    # the sum of `width` equal values of 8 or 11 bits is exact in 32 bits, so its quotient by
    # the width is that value, the differences are 0 and y is the bias
    rng = np.random.default_rng(width)
    c = draw(rng, (200, 1), dtype, 300.0)
    x = c.expand(200, width).contiguous().cuda()
    w = draw(rng, width, "f32", 0.1, 1.0).cuda()
    b = draw(rng, width, dtype, 0.1).float().cuda()
    y, mean, rstd = cuda_lib.layernorm_fwd(x, w, b)
    assert torch.equal(mean, c[:, 0].float().cuda())
    assert torch.equal(y, b.to(TORCH[dtype]).expand(200, width))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6, atol=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [128, 1032, 2048, 5120])
@pytest.mark.parametrize("xs,ds", [(1e16, 1e-12), (1e14, 1e-15), (1e-12, 1e12)])
def test_scales_far_apart(cuda_lib, width, dtype, xs, ds):
    # dx scales with ds / xs, within the format's range; nothing on the way may
    # leave fp32's (a product of two rstd would)
    rng = np.random.default_rng(width)
    x, dy, w, b = _case(rng, 37, width, dtype)
    _check(cuda_lib, x * xs, dy * ds, w, b, eps=0.0)
