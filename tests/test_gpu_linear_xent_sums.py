"""Long sums of the linear cross entropy on the GPU: the logits of its backward
at wide rows, dW over many rows, logits without a rounding."""
import numpy as np
import pytest
import torch

from ends_util import U32, assert_close, draw, f64

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half a step, relative


def _acc(n):
    """A sum of n products in the tensor cores' accumulator, 16 at a time,
    truncated to 2^-23 of the largest term, relative to the terms."""
    return (n / 16 + 17) * 4 * U32


@pytest.mark.parametrize("dtype,width,z,softcap", [
    ("f16", 16384, 30.0, 0.0), ("f16", 16384, 30.0, 50.0), ("f16", 4104, 100.0, 0.0), ("f16", 1032, 30.0, 0.0),
    ("bf16", 16384, 200.0, 0.0), ("bf16", 2048, 100.0, 60.0)])
@pytest.mark.parametrize("rows", [3, 40])
def test_backward_s_probabilities_are_the_forward_s(cuda_lib, rows, dtype, width, z, softcap):
    # every word has the same row of w, its terms of one sign (what the tensor cores
    # cut off adds up), and a 1 in a column where x is 0: that column of dx is
    # dnll * (sum_v p_v - 1) ds/dz, exactly 0.  Logits that are not those that lse was
    # made of give all probabilities the same factor, which it would show
    rng = np.random.default_rng(width + rows)
    vocab = 300
    x = np.abs(rng.standard_normal((rows, width))) + 0.25
    x[:, 0] = 0.0
    row = np.abs(rng.standard_normal(width)) + 0.25
    row *= z / (x @ row).mean()
    row[0] = 1.0
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    x = torch.from_numpy(x).to(dt).cuda()
    w = torch.from_numpy(np.tile(row, (vocab, 1))).to(dt).cuda()
    t = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    g = draw(rng, rows, "f32", 0.1, 1.0).cuda()
    _, lse = cuda_lib.linear_xent_fwd(x, w, t, softcap)
    dx, _ = cuda_lib.linear_xent_bwd(x, w, t, lse, g, softcap)
    zr = float((f64(x) @ f64(w[0])).max())
    # sum |dz| <= 2 dnll: one rounding of each (the target's is made up for, to its
    # square), exp2 (2 units in the last place), its argument, lse's sums and its
    # own rounding; the products with the column of ones
    err = U[dtype] + U[dtype] ** 2 + (4 + 120 + 64 + 8) * U32 + 2 * U32 * zr + 2 * _acc(vocab)
    if softcap:   # the slopes of the target's logit and the others', 2 / cap apart for each 1 between them
        err += 2 / softcap * zr * (_acc(min(width, 1024)) + 64 * 2.0 ** -26) + 16 * U32
    assert_close(dx[:, 0], np.zeros(rows), f64(g) * err, "dx")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dw_of_many_rows(cuda_lib, dtype):
    # w = 0: every probability is 1 / 256, dz is exact in either format, and so dw's
    # error is that of its sum over 2^19 rows (terms of one sign) and its rounding
    rng = np.random.default_rng(1)
    rows, width, vocab, g = 1 << 19, 64, 256, 2.0 ** -4
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    x = torch.from_numpy((0.5 + rng.random((rows, width))).astype(np.float32)).to(dt).cuda()
    w = torch.zeros(vocab, width, dtype=dt, device="cuda")
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
    _, dw = cuda_lib.linear_xent_bwd(x, w, t, lse, torch.full_like(nll, g), want_dx=False)
    want = np.tile(g / 256 * f64(x.double().sum(0)), (vocab, 1))
    want[0] *= -255.0
    # segments of 16384 rows, 32 of them added up with rounding
    assert_close(dw, want, (_acc(16384) + 32 * U32) * np.abs(want), "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("width", [1024, 1544, 4096])
def test_logits_whose_sums_are_exact(cuda_lib, width, dtype):
    # one element of x: a logit is one product, nothing is cut off, and the factor made
    # for sums that are (64 additions of 2^-26 at most) is the error, up to 1e-4 here
    rng = np.random.default_rng(width)
    rows, vocab = 50, 400
    w = draw(rng, (vocab, width), dtype)
    x = torch.zeros(rows, width, dtype=w.dtype)
    x[torch.arange(rows), torch.from_numpy(rng.integers(0, width, rows))] = torch.linspace(1, 40, rows).to(w.dtype)
    t = rng.integers(0, vocab, rows)
    nll, lse = cuda_lib.linear_xent_fwd(x.cuda(), w.cuda(), torch.from_numpy(t).cuda())
    z = f64(x) @ f64(w).T
    top = z.max(1, keepdims=True)
    want = np.log(np.exp(z - top).sum(1)) + top[:, 0]
    # the factor, and the roundings of the sums (as the tests of the losses have them)
    err = 64 * 2.0 ** -26 * np.abs(z).max(1) + (4 + 120 + 64) * U32 + 2 * U32 * np.abs(want)
    assert_close(lse, want, err, "lse")
    loss = want - z[np.arange(rows), t]
    assert_close(nll, loss, 2 * err + U32 * loss, "nll")
