"""After a wait that ran out, every output of the linear cross entropy on that device
is NaN.  The flag such a wait sets is set by a test entry; no wait runs out here."""
import numpy as np
import pytest
import torch

from ends_util import bits
from test_gpu_linear_xent import _case

pytestmark = pytest.mark.gpu


@pytest.fixture
def set_flag(cuda_lib):
    def f(on):
        torch.cuda.synchronize()
        cuda_lib.rn_test_set_wait_failed(on)
        torch.cuda.synchronize()
    yield f
    f(False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,width,vocab,ignored", [
    (300, 72, 1000, 0.2), (1, 512, 257, 0.0), (50, 256, 300, 2.0), (8192, 64, 40000, 0.1)])
def test_every_output_is_nan(cuda_lib, set_flag, rows, width, vocab, ignored, dtype):
    # 72: dw leaves by TMA; 2.0: every row ignored; 40000 words: two pieces
    rng = np.random.default_rng(rows)
    x, w, t, g = (v.cuda() for v in _case(rng, rows, width, vocab, dtype, ignored=ignored))
    nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
    dx, dw = cuda_lib.linear_xent_bwd(x, w, t, lse, g)
    set_flag(True)
    bad = [*cuda_lib.linear_xent_fwd(x, w, t), *cuda_lib.linear_xent_bwd(x, w, t, lse, g),
           cuda_lib.linear_xent_bwd(x, w, t, lse, g, want_dw=False)[0],
           cuda_lib.linear_xent_bwd(x, w, t, lse, g, want_dx=False)[1]]
    set_flag(False)
    for name, b in zip(("nll", "lse", "dx", "dw", "dx alone", "dw alone"), bad):
        assert bool(torch.isnan(b).all()), name
    n2, l2 = cuda_lib.linear_xent_fwd(x, w, t)
    dx2, dw2 = cuda_lib.linear_xent_bwd(x, w, t, l2, g)
    for a, b in ((nll, n2), (lse, l2), (dx, dx2), (dw, dw2)):
        assert torch.equal(bits(a), bits(b))
