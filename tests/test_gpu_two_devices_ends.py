"""The layer norm, the embedding and the linear cross entropy on cuda:1 while
cuda:0 is current, and on tensors of both: the same bits.  Skipped with one GPU."""
import numpy as np
import pytest
import torch

from ends_util import bits, draw

pytestmark = pytest.mark.gpu


def test_other_device_than_the_current_one(cuda_lib):
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")
    rng = np.random.default_rng(0)
    x, dy = draw(rng, (500, 5120), "bf16"), draw(rng, (500, 5120), "bf16")
    w, t = draw(rng, 5120, "f32", 0.1, 1.0), draw(rng, (700, 5120), "bf16", 0.02)
    ids = torch.from_numpy(rng.integers(0, 700, 500))
    outs = []
    for dev in ("cuda:0", "cuda:1"):
        a, b, c, e, i = (v.to(dev) for v in (x, dy, w, t, ids))
        y, mean, rstd = cuda_lib.layernorm_fwd(a, c)
        dx, dw, db = cuda_lib.layernorm_bwd(a, c, b, mean, rstd)
        nll, lse = cuda_lib.linear_xent_fwd(a, e, i)
        gx, gw = cuda_lib.linear_xent_bwd(a, e, i, lse, torch.ones_like(lse))
        outs.append((y, dx, dw, db, nll, gx, gw, cuda_lib.embed_fwd(i, e, 3.0), cuda_lib.embed_bwd(i, b, 700)))
        torch.cuda.synchronize(dev)
    for p, q in zip(*outs):
        assert torch.equal(bits(p.cpu()), bits(q.cpu()))
