"""The linear cross entropy on the GPU against the fp64 formulas: losses and
gradients at ragged sizes, ignored rows, the soft cap, row invariance."""
import numpy as np
import pytest
import torch

from ends_util import U32, assert_close, bits, draw, f64
from oracle.xent import linear_xent

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half a step, relative


def _case(rng, rows, width, vocab, dtype, ignored=0.2, spread=2.0):
    w = draw(rng, (vocab, width), dtype, spread / np.sqrt(width))
    target = rng.integers(0, vocab, rows)
    wt = f64(w)[target]
    x = rng.standard_normal((rows, width)) + 4 * rng.random((rows, 1)) * wt / np.linalg.norm(wt, axis=1, keepdims=True)
    x = torch.from_numpy(x.astype(np.float32)).to(w.dtype)
    target[rng.random(rows) < ignored] = [-100, vocab, -1, 2 ** 40][rows % 4]
    dnll = draw(rng, rows, "f32", 0.5, 1.0)
    return x, w, torch.from_numpy(target), dnll


def _check(rn, x, w, target, dnll, softcap, dtype, target_exact=False):
    d = [t.cuda() for t in (x, w, target, dnll)]
    nll, lse = rn.linear_xent_fwd(d[0], d[1], d[2], softcap)
    dx, dw = rn.linear_xent_bwd(d[0], d[1], d[2], lse, d[3], softcap)
    x64, w64, t, g = f64(x), f64(w), target.numpy(), f64(dnll)
    rnll, rlse, rdx, rdw, dz = linear_xent(x64, w64, t, g, softcap)
    kept = (t >= 0) & (t < w.shape[0])
    width, vocab = x.shape[1], w.shape[0]
    # the tensor cores add 16 products at a time to the accumulator; truncation
    # (2^-23 of the largest term) is allowed for in place of rounding
    acc = lambda n: (n / 16 + 17) * 4 * U32
    zerr = acc(width) * (np.abs(x64) @ np.abs(w64).T).max(1)
    zerr = zerr + (0 if not softcap else 16 * U32 * softcap)
    # exp2 within 2 units in the last place, its argument's product and
    # difference rounded (|s - max| up to 40), sums of 256 and trees, one log
    stat = (2 * 2 + 2 * 60 + 64) * U32
    serr = zerr + stat + 2 * U32 * np.abs(rlse)
    assert_close(lse, rlse, serr, "lse")
    assert_close(nll, rnll, np.where(kept, serr + zerr + U32 * np.abs(rnll), 0.0), "nll")
    assert np.all(f64(nll)[~kept] == 0.0)
    # dz: relative errors of the probability and one rounding to the format
    perr = (2 * zerr + 2 * serr + stat + 8 * U32)[:, None]
    prob = np.abs(dz) + 0.0
    prob[np.arange(len(t))[kept], t[kept]] += np.abs(g[kept]) + np.abs(dz[np.arange(len(t))[kept], t[kept]])
    tiny = 2.0 ** -24 * 2.0 ** -15 * np.abs(g).max() if dtype == "f16" else 2.0 ** -134
    dzerr = (perr * prob + U[dtype] * (np.abs(dz) + perr * prob) + tiny * 2) * kept[:, None]
    if target_exact:   # the target's dz enters the sums with its rounding's rest, rounded itself
        i, j = np.arange(len(t))[kept], t[kept]
        dzerr[i, j] = (perr * prob)[i, j] + U[dtype] ** 2 * (np.abs(dz)[i, j] + (perr * prob)[i, j]) + tiny * 2
    assert_close(dx, rdx, dzerr @ np.abs(w64) + (acc(vocab) + 40 * U32) * (np.abs(dz) @ np.abs(w64)), "dx")
    xk = np.where(kept[:, None], np.abs(x64), 0.0)
    assert_close(dw, rdw, dzerr.T @ xk + (acc(len(t)) + 2 * U32) * (np.abs(dz).T @ xk), "dw")
    return nll, lse, dx, dw


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,width,vocab", [
    (1, 8, 1), (1, 64, 257), (3, 72, 1000), (130, 128, 255), (257, 136, 513), (64, 2048, 4099),
    (300, 1032, 2001), (7, 512, 40001), (513, 264, 16385), (256, 256, 256)])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_losses_and_gradients(cuda_lib, rows, width, vocab, softcap, dtype):
    rng = np.random.default_rng(rows + vocab)
    _check(cuda_lib, *_case(rng, rows, width, vocab, dtype), softcap, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,width,vocab,ignored,softcap", [
    (1, 264, 3000, 0.0, 0.0), (3, 1048, 2500, 0.0, 9.0), (32, 128, 17000, 0.0, 0.0), (300, 72, 500, 0.9, 4.0)])
def test_few_rows_keep_the_target_s_gradient(cuda_lib, rows, width, vocab, ignored, softcap, dtype):
    # up to 32 rows with a loss: the rounding of the target's dz, which few rows do
    # not average out, is made up for in dx and dw
    rng = np.random.default_rng(rows)
    case = _case(rng, rows, width, vocab, dtype, ignored=ignored)
    assert 0 < int(((case[2] >= 0) & (case[2] < vocab)).sum()) <= 32
    _check(cuda_lib, *case, softcap, dtype, target_exact=True)


def test_confident_targets_in_wide_rows(cuda_lib):
    # a target's logit of 25 from 4096 products: what the tensor cores cut off it
    # (1e-5) is not in its loss of 1e-7 to 1e-2
    rng = np.random.default_rng(12)
    width, vocab = 4096, 400
    w = draw(rng, (vocab, width), "bf16", 1 / 64)
    t = rng.integers(0, vocab, 24)
    wt = f64(w)[t]
    x = torch.from_numpy((wt / (wt ** 2).sum(1, keepdims=True) * np.linspace(12, 25, 24)[:, None]).astype(np.float32)).bfloat16()
    nll, _ = cuda_lib.linear_xent_fwd(x.cuda(), w.cuda(), torch.from_numpy(t).cuda())
    want, _ = linear_xent(f64(x), f64(w), t)
    # the target's logit: 4096 products of fp32, 64 to a lane's two sums, 6 joins
    # (38 U32 of the terms); the others' cut-off moves a loss relative to itself
    zt = 38 * U32 * (np.abs(f64(x)) * np.abs(wt)).sum(1)
    others = (4096 / 16 + 17) * 4 * U32 * (np.abs(f64(x)) @ np.abs(f64(w)).T).max(1)
    assert_close(nll, want, zt * np.minimum(1, 2 * want) + (others + 300 * U32) * want * 2 + 50 * U32, "nll")


@pytest.mark.parametrize("rows,width,vocab", [(5, 16384, 300), (9, 2056, 20001), (600, 1600, 9000)])
def test_several_segments_of_the_width(cuda_lib, rows, width, vocab):
    # K in segments of 1024, the last one short, few tiles and several
    # to a pair of CTAs
    rng = np.random.default_rng(0)
    _check(cuda_lib, *_case(rng, rows, width, vocab, "bf16"), 0.0, "bf16")


@pytest.mark.parametrize("rows", [1, 200])
def test_every_row_ignored(cuda_lib, rows):
    rng = np.random.default_rng(1)
    x, w, t, g = _case(rng, rows, 256, 700, "bf16", ignored=2.0)
    nll, _, dx, dw = _check(cuda_lib, x, w, t, g, 0.0, "bf16")
    assert not bool(dx.any()) and not bool(dw.any()) and not bool(nll.any())


def test_ignored_rows_take_no_part_whatever_they_hold(cuda_lib):
    rng = np.random.default_rng(2)
    x, w, t, g = _case(rng, 333, 264, 3001, "bf16", ignored=0.4)
    gone = (t < 0) | (t >= 3001)
    assert 0 < int(gone.sum()) < 333
    _, lse = cuda_lib.linear_xent_fwd(x.cuda(), w.cuda(), t.cuda())
    dx, dw = cuda_lib.linear_xent_bwd(x.cuda(), w.cuda(), t.cuda(), lse, g.cuda())
    x2, g2, l2 = x.clone(), g.clone(), lse.cpu().clone()
    x2[gone], g2[gone], l2[gone] = float("nan"), float("inf"), float("nan")
    dx2, dw2 = cuda_lib.linear_xent_bwd(x2.cuda(), w.cuda(), t.cuda(), l2.cuda(), g2.cuda())
    assert torch.equal(bits(dx), bits(dx2)) and torch.equal(bits(dw), bits(dw2))
    nll2, _ = cuda_lib.linear_xent_fwd(x2.cuda(), w.cuda(), t.cuda())
    assert not bool(nll2[gone.cuda()].any()) and bool(torch.isfinite(nll2).all())


def test_confident_targets_keep_their_small_loss(cuda_lib):
    # the target's logit stands out by 3 to 60: losses from 0.1 down to zero,
    # each relative to itself (no cancellation against the log-sum-exp)
    width, vocab = 64, 500
    w = torch.zeros(vocab, width)
    w[7, 0] = 1.0
    x = torch.zeros(58, width)
    x[:, 0] = torch.arange(3, 61)
    t = torch.full((58,), 7)
    nll, lse = cuda_lib.linear_xent_fwd(x.bfloat16().cuda(), w.bfloat16().cuda(), t.cuda())
    z = np.arange(3, 61, dtype=np.float64)
    want = np.log1p((vocab - 1) * np.exp(-z))
    # log(1 + e) of the fp32 sum.  From the target's term, 1, on, every addition
    # rounds a partial sum in [1, 2) by U32 * 2 at most where it stays below 2:
    # 8 in its accumulator of the 32-column chunk, 2 to join the accumulators, 8
    # chunks, 1 + 3 tiles and groups = 22, and the terms' own relative errors
    assert_close(nll, want, 200 * U32 * np.minimum(want, 1) + 22 * 2 * U32, "nll")
    # fp16 gradients of a likely target stay relative to themselves too
    g = torch.ones(58)
    dx, _ = cuda_lib.linear_xent_bwd(x.half().cuda(), w.half().cuda(), t.cuda(), lse, g.cuda())
    p = (vocab - 1) * np.exp(-z) / (1 + (vocab - 1) * np.exp(-z))
    err = np.zeros((58, width))
    err[:, 0] = p * 2.0 ** -10 + 64 * U32
    wantdx = np.zeros((58, width))
    wantdx[:, 0] = -p
    assert_close(dx, wantdx, err, "dx")


def test_pieces_of_the_vocabulary_and_row_invariance(cuda_lib):
    # 8192 rows x 40000: three chunks in two pieces; 200 rows: one
    # piece.  nll, lse and dx of a row are the same bits; dw against fp64
    rng = np.random.default_rng(3)
    rows, width, vocab = 8192, 128, 40000
    x, w, t, g = (v.cuda() for v in _case(rng, rows, width, vocab, "bf16"))
    nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
    dx, dw = cuda_lib.linear_xent_bwd(x, w, t, lse, g)
    for lo, hi in ((0, 200), (5, 6), (4001, 4300)):
        n2, l2 = cuda_lib.linear_xent_fwd(x[lo:hi].contiguous(), w, t[lo:hi].contiguous())
        assert torch.equal(bits(n2), bits(nll[lo:hi])) and torch.equal(bits(l2), bits(lse[lo:hi]))
        d2, _ = cuda_lib.linear_xent_bwd(x[lo:hi].contiguous(), w, t[lo:hi].contiguous(), l2,
                                         g[lo:hi].contiguous(), want_dw=False)
        assert torch.equal(bits(d2), bits(dx[lo:hi]))
    z = x.double() @ w.double().T
    d = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    kept = (t >= 0) & (t < vocab)
    d[torch.arange(rows, device="cuda")[kept], t[kept]] -= 1.0
    d *= torch.where(kept, g.double(), 0.0)[:, None]
    want = d.T @ x.double()
    bound = (2.0 ** -8 + (rows / 16 + 17) * 4 * U32 + 2e-4) * (d.abs().T @ x.double().abs())
    assert_close(dw, f64(want), f64(bound), "dw")
    dx2, dw2 = cuda_lib.linear_xent_bwd(x, w, t, lse, g)
    assert torch.equal(bits(dx), bits(dx2)) and torch.equal(bits(dw), bits(dw2))
    # one gradient only: the same bits
    only_w = cuda_lib.linear_xent_bwd(x, w, t, lse, g, want_dx=False)
    assert only_w[0] is None and torch.equal(bits(only_w[1]), bits(dw))


@pytest.mark.parametrize("softcap", [0.75, 1e5])
def test_caps_far_below_and_above_the_logits(cuda_lib, softcap):
    # 0.75: most logits saturate; 1e5: tanh(z / cap) of tiny arguments, z again but
    # for roundings relative to itself
    rng = np.random.default_rng(11)
    x, w, t, g = _case(rng, 60, 128, 700, "bf16")
    if softcap < 1:
        _check(cuda_lib, x, w, t, g, softcap, "bf16")
        return
    d = [v.cuda() for v in (x, w, t)]
    nll, lse = cuda_lib.linear_xent_fwd(*d, softcap)
    want, wlse = linear_xent(f64(x), f64(w), t.numpy(), None, softcap)
    zmax = np.abs(f64(x) @ f64(w).T).max(1)
    # the logits' own error (acc, as in _check), then the quotient, the series'
    # four roundings and the product: 8 U32 relative to the logit
    err = (128 / 16 + 17) * 4 * U32 * (np.abs(f64(x)) @ np.abs(f64(w)).T).max(1) + 8 * U32 * zmax
    assert_close(lse, wlse, err + 200 * U32 + 2 * U32 * np.abs(wlse), "lse")
    kept = (t.numpy() >= 0) & (t.numpy() < 700)
    assert_close(nll, want, np.where(kept, 2 * err + 200 * U32 + 2 * U32 * np.abs(wlse), 0), "nll")


@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_logits_of_minus_infinity(cuda_lib, softcap):
    # words that a row of w makes impossible: a whole block of 128 columns, the
    # last ones, single ones (with a cap they stand at its lower end)
    rng = np.random.default_rng(13)
    vocab, width = 700, 136
    x, w, t, _ = _case(rng, 40, width, vocab, "bf16")
    x[:, 0] = 1.0
    wz = w.clone()
    gone = np.zeros(vocab, bool)
    gone[[3, 300]] = gone[128:256] = gone[620:] = True
    wz[torch.from_numpy(gone), 0] = float("-inf")
    d = [v.cuda() for v in (x, wz, t)]
    nll, lse = cuda_lib.linear_xent_fwd(*d, softcap)
    kept = (t.numpy() >= 0) & (t.numpy() < vocab)
    hit = kept & gone[np.where(kept, t.numpy(), 0)]
    z = f64(x) @ f64(w).T
    s = np.where(gone, -np.inf, z) if not softcap else softcap * np.where(gone, -1.0, np.tanh(z / softcap))
    wlse = np.log(np.exp(s - s.max(1, keepdims=True)).sum(1)) + s.max(1)
    want = np.where(kept, wlse - s[np.arange(40), np.where(kept, t.numpy(), 0)], 0.0)
    # as in _check
    zerr = (width / 16 + 17) * 4 * U32 * (np.abs(f64(x)) @ np.abs(f64(w)).T).max(1) + 16 * U32 * softcap
    serr = zerr + (4 + 120 + 64) * U32 + 2 * U32 * np.abs(wlse)
    assert_close(lse, wlse, serr, "lse")
    fin = np.isfinite(want)
    assert hit.any() and (softcap or not fin[hit].any())
    got = nll.cpu()
    assert bool(torch.isposinf(got[torch.from_numpy(~fin)]).all())
    assert_close(got[torch.from_numpy(fin)], want[fin], np.where(kept, serr + zerr + U32 * np.abs(np.where(fin, want, 0)), 0.0)[fin], "nll")


def test_many_rows_with_a_loss_here_and_there(cuda_lib):
    # several blocks of rows to a CTA of the packing kernel, kept rows in clumps:
    # the same as the kept rows alone, bitwise
    rng = np.random.default_rng(10)
    rows, width, vocab = 90001, 64, 300
    x, w, t, g = _case(rng, rows, width, vocab, "bf16", ignored=0.0)
    keep = np.repeat(rng.random(rows // 50 + 1) < 0.1, 50)[:rows]
    keep[[0, rows - 1]] = True
    t = torch.where(torch.from_numpy(keep), t, torch.tensor(-100))
    x, w, t, g, k = (v.cuda() for v in (x, w, t, g, torch.from_numpy(keep)))
    _, lse = cuda_lib.linear_xent_fwd(x, w, t)
    dx, dw = cuda_lib.linear_xent_bwd(x, w, t, lse, g)
    dx2, dw2 = cuda_lib.linear_xent_bwd(x[k].contiguous(), w, t[k].contiguous(), lse[k].contiguous(), g[k].contiguous())
    assert torch.equal(bits(dx[k]), bits(dx2)) and not bool(dx[~k].any()) and torch.equal(bits(dw), bits(dw2))


def test_no_rows(cuda_lib):
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(300, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    e = torch.zeros(0, device="cuda")
    nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
    dx, dw = cuda_lib.linear_xent_bwd(x, w, t, lse, e)
    assert nll.numel() == 0 and dx.shape == (0, 64) and dw.shape == w.shape and not bool(dw.any())


def test_writes_only_its_outputs(cuda_lib):
    rng = np.random.default_rng(5)
    rows, width, vocab, guard = 67, 72, 301, 64
    x, w, t, g = (v.cuda() for v in _case(rng, rows, width, vocab, "f16"))
    lib = cuda_lib.load()
    wsb = [int(lib.linear_xent_fwd_workspace_bytes(rows, vocab)), int(lib.linear_xent_bwd_workspace_bytes(rows, width, vocab))]
    raws, outs = [], []
    for n, dt in ((rows, torch.float32), (rows, torch.float32), (rows * width, torch.float16),
                  (vocab * width, torch.float16), (wsb[0], torch.uint8), (wsb[1], torch.uint8)):
        raw = torch.full((n + 2 * guard,), 7, dtype=dt, device="cuda")
        raws.append(raw)
        outs.append(raw[guard:guard + n])
    cuda_lib.linear_xent_fwd(x, w, t, nll=outs[0], lse=outs[1], ws=outs[4])
    cuda_lib.linear_xent_bwd(x, w, t, outs[1], g, dx=outs[2].view(rows, width), dw=outs[3].view(vocab, width), ws=outs[5])
    for raw in raws:
        assert bool((raw[:guard] == 7).all()) and bool((raw[-guard:] == 7).all())
    nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
    dx, dw = cuda_lib.linear_xent_bwd(x, w, t, lse, g)
    for got, want in zip(outs, (nll, lse, dx, dw)):
        assert torch.equal(bits(got), bits(want.reshape(-1)))


@pytest.mark.parametrize("width", [72, 256])
def test_buffers_on_16_bytes_only(cuda_lib, width):
    # every pointer 16 bytes past a 256-byte boundary: the same bits
    rng = np.random.default_rng(9)
    rows, vocab = 70, 900
    x, w, t, g = (v.cuda() for v in _case(rng, rows, width, vocab, "bf16"))
    nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
    dx, dw = cuda_lib.linear_xent_bwd(x, w, t, lse, g)

    def shifted(n, dt):
        return torch.empty(n + 16, dtype=dt, device="cuda")[16 // torch.empty(0, dtype=dt).element_size():][:n]

    x2, w2 = shifted(rows * width, x.dtype).view(rows, width), shifted(vocab * width, x.dtype).view(vocab, width)
    x2.copy_(x)
    w2.copy_(w)
    lib = cuda_lib.load()
    ws = shifted(int(lib.linear_xent_bwd_workspace_bytes(rows, width, vocab)), torch.uint8)
    n2, l2 = cuda_lib.linear_xent_fwd(x2, w2, t, ws=ws)
    dx2, dw2 = cuda_lib.linear_xent_bwd(x2, w2, t, l2, g, dx=shifted(rows * width, x.dtype).view(rows, width),
                                        dw=shifted(vocab * width, x.dtype).view(vocab, width), ws=ws)
    for got, want in ((n2, nll), (l2, lse), (dx2, dx), (dw2, dw)):
        assert torch.equal(bits(got), bits(want))


def test_captured_and_replayed_with_other_targets(cuda_lib):
    rng = np.random.default_rng(6)
    x, w, t, g = (v.cuda() for v in _case(rng, 300, 256, 3000, "bf16", ignored=0.1))
    t2 = t.clone()
    t2[:150] = -1
    want = []
    for k in (t, t2):
        nll, lse = cuda_lib.linear_xent_fwd(x, w, k, 9.0)
        want.append((nll, lse, *cuda_lib.linear_xent_bwd(x, w, k, lse, g, 9.0)))
    buf = t.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nll, lse = cuda_lib.linear_xent_fwd(x, w, buf, 9.0)
        dx, dw = cuda_lib.linear_xent_bwd(x, w, buf, lse, g, 9.0)
    for k, i in enumerate((t, t2, t)):
        buf.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((nll, lse, dx, dw), want[k % 2]):
            assert torch.equal(bits(got), bits(ref))


def test_two_streams_at_once(cuda_lib):
    rng = np.random.default_rng(7)
    work = []
    for k in range(2):
        x, w, t, g = (v.cuda() for v in _case(rng, 500, 512, 9000, "bf16"))
        nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
        work.append((x, w, t, g, (nll, lse, *cuda_lib.linear_xent_bwd(x, w, t, lse, g))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(4):
        got = []
        for s, (x, w, t, g, _) in zip(streams, work):
            with torch.cuda.stream(s):
                nll, lse = cuda_lib.linear_xent_fwd(x, w, t)
                got.append((nll, lse, *cuda_lib.linear_xent_bwd(x, w, t, lse, g)))
        torch.cuda.synchronize()
        for out, (*_, want) in zip(got, work):
            for a, b in zip(out, want):
                assert torch.equal(bits(a), bits(b))


def test_autograd_matches_differences(cuda_lib):
    # a central difference of the fp64 loss along a random direction of x and of
    # w: its own error is O(h^2) = 1e-7; the gradients carry fp16 roundings
    rng = np.random.default_rng(8)
    x, w, t, g = _case(rng, 20, 64, 300, "f16")
    leaves = [v.cuda().requires_grad_(True) for v in (x, w)]
    nll = cuda_lib.autograd.linear_cross_entropy(*leaves, t.cuda(), 6.0)
    (nll * g.cuda()).sum().backward()
    v64 = [f64(x), f64(w)]
    for i, leaf in enumerate(leaves):
        d = rng.standard_normal(v64[i].shape)
        h = 1e-4
        up, dn = list(v64), list(v64)
        up[i], dn[i] = v64[i] + h * d, v64[i] - h * d
        loss = lambda v: float((linear_xent(*v, t.numpy(), None, 6.0)[0] * f64(g)).sum())
        want = (loss(up) - loss(dn)) / (2 * h)
        grad = f64(leaf.grad)
        # two roundings of half an fp16 step each, over every product of the sums
        assert abs(float((grad * d).sum()) - want) <= 2 ** -9 * float(np.abs(grad * d).sum()) + 2e-2
