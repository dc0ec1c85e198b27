"""A loss is minus the logarithm of a probability: never below zero."""
import numpy as np
import pytest
import torch

from ends_util import draw, f64
from oracle.xent import linear_xent

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("width", [64, 1024, 4096])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
def test_targets_up_to_certain(cuda_lib, width, softcap, dtype):
    # targets whose logits lead by up to 30, past where 32 bits tell p from 1
    rng = np.random.default_rng(width)
    rows, vocab = 2000, 700
    w = draw(rng, (vocab, width), dtype, 0.5 / np.sqrt(width))
    t = rng.integers(0, vocab, rows)
    wt = f64(w)[t]
    lead = 60 * rng.random((rows, 1)) / np.linalg.norm(wt, axis=1, keepdims=True)
    x = torch.from_numpy((rng.standard_normal((rows, width)) + lead * wt).astype(np.float32)).to(w.dtype)
    nll, lse = cuda_lib.linear_xent_fwd(x.cuda(), w.cuda(), torch.from_numpy(t).cuda(), softcap)
    assert bool((nll >= 0).all()), float(nll.min())
    want, _ = linear_xent(f64(x[:200]), f64(w), t[:200], None, softcap)
    sure = want < 2.0 ** -24
    assert sure.any() and np.all(f64(nll[:200])[sure] < 2.0 ** -22)


def test_a_loss_that_is_not_a_number_stays_one(cuda_lib):
    x = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 5] = float("nan")
    w = torch.zeros(200, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.tensor([3, 4, 5], device="cuda")
    nll, _ = cuda_lib.linear_xent_fwd(x, w, t)
    assert torch.isnan(nll).tolist() == [False, True, False]
