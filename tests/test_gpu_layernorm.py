"""Layer norm on the GPU against the fp64 formulas: values and gradients,
row invariance, masks, in-place forms, captured graphs."""
import numpy as np
import pytest
import torch

from ends_util import U32, assert_close, bits, draw, f64
from oracle.layernorm import layernorm_bwd, layernorm_fwd

pytestmark = pytest.mark.gpu

# widths of every team shape: one vector, sub-warp, warp, 4-warp, 8-, 16- and
# 32-warp teams, full and ragged
WIDTHS = [8, 16, 24, 40, 72, 128, 256, 512, 776, 1032, 2048, 5120, 6144, 8192, 10240, 16376, 16384]


def _sum_bound(n, width):
    """Longest chain of fp32 additions of a row sum: 16 elements of a vector,
    up to 5 vectors joined, 5 butterfly steps, 5 levels of warps, and the
    products' roundings."""
    return (16 + 5 + 5 + 5 + 4) * U32


def _case(rng, rows, width, dtype, biased=True, shift=0.5):
    x = draw(rng, (rows, width), dtype, shift=shift)
    dy = draw(rng, (rows, width), dtype)
    w = draw(rng, width, "f32", 0.1, 1.0)
    b = draw(rng, width, "f32", 0.1) if biased else None
    return x, dy, w, b


def _check(rn, x, dy, w, b, eps=1e-5, mask=None):
    d = lambda t: None if t is None else t.cuda()
    xd, dyd, wd, bd = d(x), d(dy), d(w), d(b)
    y, mean, rstd = rn.layernorm_fwd(xd, wd, bd, eps)
    dx, dw, db = rn.layernorm_bwd(xd, wd, dyd, mean, rstd, row_mask=d(mask),
                                  want_db=b is not None)
    x64, w64, dy64 = f64(x), f64(w), f64(dy)
    b64 = None if b is None else f64(b)
    m64 = None if mask is None else mask.numpy().astype(bool)
    ry, rmean, rrstd = layernorm_fwd(x64, w64, b64, eps)
    rdx, rdw, rdb = layernorm_bwd(x64, w64, dy64, eps, m64)
    rows, width = x64.shape
    chain = _sum_bound(rows, width)
    # mean: the sum's error, relative to the mean of |x|, and a division
    dmean = (chain + 2 * U32) * np.abs(x64).mean(1) + U32 * np.abs(rmean)
    assert_close(mean, rmean, dmean, "mean")
    # an error dm of the mean moves the variance by dm^2 at most (the sum of
    # c is zero); c itself is rounded once (relative U32 of |x| + |mean|)
    c = np.abs(x64 - rmean[:, None])
    dc = dmean[:, None] + U32 * (c + dmean[:, None])
    var = 1.0 / rrstd ** 2
    dvar = dmean ** 2 + (chain + 4 * U32) * (c * c).mean(1) + 2 * (U32 * c * c).mean(1) + U32 * var
    drstd = rrstd * (0.5 * dvar / var + 4 * U32)     # rsqrtf: 2 units in the last place
    assert_close(rstd, rrstd, drstd, "rstd")
    rel = (drstd / rrstd)[:, None]
    # xh = c * rstd; y = xh * w + b
    r = rrstd[:, None]
    dxh = r * (dc + c * (rel + U32))
    dy_err = np.abs(w64) * (dxh + 2 * U32 * c * r) + (0 if b64 is None else U32 * np.abs(ry))
    assert_close(y, ry, dy_err, "y")
    # dx = rstd * (g - m1 - xh * m2)
    g, xh = np.abs(w64 * dy64), c * r
    m1, m2 = g.mean(1)[:, None], (g * xh).mean(1)[:, None]
    dm1 = (chain + 4 * U32) * m1
    dm2 = (chain + 6 * U32) * m2 + (g * dxh).mean(1)[:, None]
    terms = g + m1 + xh * m2
    ddx = r * (4 * U32 * terms + dm1 + dxh * m2 + xh * dm2 + rel * terms)
    assert_close(dx, rdx, ddx, "dx")
    # dw, db: a team's rows one after the other, then trees (at most 20 levels)
    keep = np.ones(rows, bool) if m64 is None else m64
    seq = (rows / 148 + 8 + 20) * U32
    tw = (np.abs(dy64) * xh)[keep].sum(0)
    assert_close(dw, rdw, seq * tw + (np.abs(dy64) * dxh)[keep].sum(0) + 2 * U32 * tw, "dw")
    if b is not None:
        assert_close(db, rdb, seq * np.abs(dy64)[keep].sum(0), "db")
    else:
        assert db is None
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_values_and_gradients(cuda_lib, width, dtype):
    rng = np.random.default_rng(width)
    for rows in (1, 2, 67) if width > 5000 else (1, 3, 259):
        _check(cuda_lib, *_case(rng, rows, width, dtype, biased=rows != 3))


@pytest.mark.parametrize("rows,width,dtype", [(5003, 128, "bf16"), (2049, 2048, "f16"),
                                              (1200, 4096, "bf16"), (4001, 40, "f32")])
def test_many_rows(cuda_lib, rows, width, dtype):
    rng = np.random.default_rng(rows)
    _check(cuda_lib, *_case(rng, rows, width, dtype))


def test_large_mean_does_not_cancel(cuda_lib):
    rng = np.random.default_rng(5)
    _check(cuda_lib, *_case(rng, 33, 2048, "f32", shift=1000.0))


def test_constant_rows_and_zero_eps_free_input(cuda_lib):
    # a constant row has variance zero: y is the bias, rstd 1 / sqrt(eps)
    x = torch.full((4, 256), 3.0, device="cuda")
    w, b = torch.ones(256, device="cuda"), torch.full((256,), 0.25, device="cuda")
    y, mean, rstd = cuda_lib.layernorm_fwd(x, w, b, 1e-6)
    assert torch.equal(mean, torch.full((4,), 3.0, device="cuda"))
    assert torch.equal(y, torch.full_like(x, 0.25))
    assert torch.allclose(rstd, torch.full((4,), 1e3, device="cuda"), rtol=1e-6)


@pytest.mark.parametrize("rows,width,dtype", [(37, 128, "bf16"), (300, 1032, "bf16"), (70, 5120, "f16")])
def test_row_mask_leaves_rows_out_whatever_they_hold(cuda_lib, rows, width, dtype):
    rng = np.random.default_rng(width)
    x, dy, w, b = _case(rng, rows, width, dtype)
    mask = torch.from_numpy(rng.random(rows) < 0.6)
    _, _, _, _, dw, db = _check(cuda_lib, x, dy, w, b, mask=mask)
    x2, dy2 = x.clone(), dy.clone()
    x2[~mask] = float("nan")
    dy2[~mask] = float("inf")
    xd, dyd, wd = x2.cuda(), dy2.cuda(), w.cuda()
    _, mean, rstd = cuda_lib.layernorm_fwd(xd, wd, b.cuda())
    _, dw2, db2 = cuda_lib.layernorm_bwd(xd, wd, dyd, mean, rstd, row_mask=mask.cuda())
    assert torch.equal(bits(dw), bits(dw2)) and torch.equal(bits(db), bits(db2))


def test_no_rows_and_no_selected_row_give_the_empty_sum(cuda_lib):
    w = torch.ones(136, device="cuda")
    neg0 = torch.full((136,), -0.0, device="cuda")
    for rows in (0, 9):
        x = torch.randn(rows, 136, device="cuda")
        y, mean, rstd = cuda_lib.layernorm_fwd(x, w)
        assert y.shape == x.shape and mean.numel() == rows
        mask = torch.zeros(rows, dtype=torch.bool, device="cuda")
        _, dw, db = cuda_lib.layernorm_bwd(x, w, x.clone(), mean, rstd, row_mask=mask)
        assert torch.equal(bits(dw), bits(neg0)) and torch.equal(bits(db), bits(neg0))


@pytest.mark.parametrize("width,dtype", [(128, "bf16"), (1032, "f16"), (5120, "bf16"), (8192, "f32")])
def test_rows_alone_and_in_any_batch_agree_bitwise(cuda_lib, width, dtype):
    rng = np.random.default_rng(1)
    x, dy, w, b = (t.cuda() for t in _case(rng, 150, width, dtype))
    y, mean, rstd = cuda_lib.layernorm_fwd(x, w, b)
    dx, _, _ = cuda_lib.layernorm_bwd(x, w, dy, mean, rstd)
    for lo, hi in ((0, 1), (7, 8), (149, 150), (3, 90)):
        ys, ms, rs = cuda_lib.layernorm_fwd(x[lo:hi].contiguous(), w, b)
        dxs, _, _ = cuda_lib.layernorm_bwd(x[lo:hi].contiguous(), w, dy[lo:hi].contiguous(), ms, rs)
        for got, want in ((ys, y), (ms, mean), (rs, rstd), (dxs, dx)):
            assert torch.equal(bits(got), bits(want[lo:hi]))


def test_repeated_runs_and_streams_give_the_same_bits(cuda_lib):
    rng = np.random.default_rng(2)
    x, dy, w, b = (t.cuda() for t in _case(rng, 3000, 1024, "bf16"))
    _, mean, rstd = cuda_lib.layernorm_fwd(x, w, b)
    _, dw, db = cuda_lib.layernorm_bwd(x, w, dy, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((int(cuda_lib.load().layernorm_bwd_workspace_bytes(3000, 1024, 1)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    _, dw2, db2 = cuda_lib.layernorm_bwd(x, w, dy, mean, rstd, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(bits(dw), bits(dw2)) and torch.equal(bits(db), bits(db2))


def test_in_place_forms(cuda_lib):
    rng = np.random.default_rng(3)
    x, dy, w, b = (t.cuda() for t in _case(rng, 500, 776, "bf16"))
    y, mean, rstd = cuda_lib.layernorm_fwd(x, w, b)
    dx, dw, db = cuda_lib.layernorm_bwd(x, w, dy, mean, rstd)
    x2, dy2 = x.clone(), dy.clone()
    dx2, dw2, _ = cuda_lib.layernorm_bwd(x2, w, dy2, mean, rstd, dx=dy2)
    y2, _, _ = cuda_lib.layernorm_fwd(x2, w, b, y=x2)
    assert y2 is x2 and torch.equal(bits(y2), bits(y))
    assert dx2 is dy2 and torch.equal(bits(dx2), bits(dx)) and torch.equal(bits(dw2), bits(dw))


def test_captured_and_replayed(cuda_lib):
    rng = np.random.default_rng(4)
    x, dy, w, b = (t.cuda() for t in _case(rng, 700, 2048, "bf16"))
    y, mean, rstd = cuda_lib.layernorm_fwd(x, w, b)
    dx, dw, db = cuda_lib.layernorm_bwd(x, w, dy, mean, rstd)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cy, cm, cr = cuda_lib.layernorm_fwd(x, w, b)
        cdx, cdw, cdb = cuda_lib.layernorm_bwd(x, w, dy, cm, cr)
    for _ in range(2):
        for t in (cy, cdx, cdw, cdb):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for got, want in ((cy, y), (cdx, dx), (cdw, dw), (cdb, db)):
            assert torch.equal(bits(got), bits(want))


def test_autograd_gradients_match_differences(cuda_lib):
    # central differences of the fp64 forward along random directions against
    # the fp32 gradients: the difference quotient's error is O(h^2), 1e-8 here
    rng = np.random.default_rng(6)
    x, dy, w, b = _case(rng, 5, 40, "f32")
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
    (cuda_lib.autograd.layer_norm(*leaves) * dy.cuda()).sum().backward()
    vals = [f64(t) for t in (x, w, b)]

    def loss(v):
        return float((layernorm_fwd(*v)[0] * f64(dy)).sum())

    for i, leaf in enumerate(leaves):
        d = rng.standard_normal(vals[i].shape)
        h = 1e-4
        up, dn = list(vals), list(vals)
        up[i], dn[i] = vals[i] + h * d, vals[i] - h * d
        want = (loss(up) - loss(dn)) / (2 * h)
        got = float((f64(leaf.grad) * d).sum())
        # 200 products, each gradient within 100 U32 of terms of size 10 at most
        assert abs(got - want) <= 200 * 100 * U32 * 10 + 1e-6
