"""The embedding and its gradient on the GPU against the fp64 sums, the runs'
fixed order, and the documented treatment of ids outside the table."""
import numpy as np
import pytest
import torch

from ends_util import U32, assert_close, bits, draw, f64
from oracle.embedding import embed_bwd, embed_fwd

pytestmark = pytest.mark.gpu


def _ids(rng, tokens, vocab, kind):
    if kind == "uniform":
        return rng.integers(0, vocab, tokens)
    if kind == "one":                       # every token the same row
        return np.full(tokens, vocab - 1)
    if kind == "few":                       # long runs beside short ones
        return np.minimum((rng.pareto(0.7, tokens)).astype(np.int64), vocab - 1)
    bad = rng.integers(-vocab, 2 * vocab, tokens)   # ids outside the table too
    bad[:: 7] = [-100, 2 ** 40, vocab, -1, -2 ** 62][tokens % 5]
    return bad


def _grad_bound(ids, dy64, vocab, scale, old=None):
    """fp32 error of the sums: 31 additions in a leaf, a tree of at most 24
    levels, the scaling."""
    mag = embed_bwd(ids, np.abs(dy64), vocab, abs(scale))
    n = np.bincount(ids[(ids >= 0) & (ids < vocab)], minlength=vocab)
    depth = np.minimum(n, 32) + np.ceil(np.log2(np.maximum(n / 32, 1))) + 1
    e = depth[:, None] * U32 * mag
    return e if old is None else e + U32 * np.abs(old)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,vocab,width,kind", [
    (1, 1, 8, "uniform"), (1, 1000, 2048, "uniform"), (31, 7, 72, "few"), (33, 2, 136, "one"),
    (64, 600, 512, "outside"), (1000, 513, 1032, "few"), (2049, 70001, 128, "uniform"),
    (5000, 300, 776, "few"), (4097, 11, 16, "one"), (700, 40, 16384, "few"), (9000, 100, 40, "outside")])
def test_values_and_gradients(cuda_lib, tokens, vocab, width, kind, dtype):
    rng = np.random.default_rng(tokens + vocab)
    ids = _ids(rng, tokens, vocab, kind)
    table, dy = draw(rng, (vocab, width), dtype), draw(rng, (tokens, width), dtype)
    scale = 1.0 if tokens == 1 else float(np.float32(np.sqrt(width)))
    i = torch.from_numpy(ids).cuda()
    y = cuda_lib.embed_fwd(i, table.cuda(), scale)
    want = embed_fwd(ids, f64(table), scale)
    assert_close(y, want, U32 * np.abs(want), "y")
    d = cuda_lib.embed_bwd(i, dy.cuda(), vocab, scale)
    assert_close(d, embed_bwd(ids, f64(dy), vocab, scale), _grad_bound(ids, f64(dy), vocab, scale), "dtable")
    old = draw(rng, (vocab, width), dtype)
    got = cuda_lib.embed_bwd(i, dy.cuda(), vocab, scale, dtable=old.cuda(), accumulate=True)
    assert_close(got, embed_bwd(ids, f64(dy), vocab, scale, f64(old)),
                 _grad_bound(ids, f64(dy), vocab, scale, f64(old)), "dtable, accumulated")
    untouched = np.setdiff1d(np.arange(vocab), ids)
    assert torch.equal(bits(got.cpu()[untouched]), bits(old[untouched]))


def test_many_tokens_and_a_long_run(cuda_lib):
    # about 20000 tokens of one id among 70000: a run of hundreds of leaves
    rng = np.random.default_rng(0)
    tokens, vocab, width = 70001, 151936, 64
    ids = np.where(rng.random(tokens) < 0.3, 77, rng.integers(0, vocab, tokens))
    dy = draw(rng, (tokens, width), "f32")
    d = cuda_lib.embed_bwd(torch.from_numpy(ids).cuda(), dy.cuda(), vocab)
    want = np.zeros((vocab, width))
    np.add.at(want, ids, f64(dy))
    mag = np.zeros((vocab, width))
    np.add.at(mag, ids, np.abs(f64(dy)))
    assert_close(d, want, (32 + 24 + 1) * U32 * mag, "dtable")


@pytest.mark.parametrize("tokens", [1024, 1025, 4095, 4096, 4097])
@pytest.mark.parametrize("vocab", [511, 512, 2 ** 18 - 1, 2 ** 18, 300007])
def test_sorts_of_few_tokens(cuda_lib, tokens, vocab):
    # one, two and three digits of nine bits; the sort of one CTA and the cluster's
    rng = np.random.default_rng(tokens + vocab)
    ids = np.where(rng.random(tokens) < 0.3, rng.integers(0, 20, tokens), rng.integers(-9, vocab, tokens))
    ids[: tokens // 3 : 2] = vocab - 1
    dy = draw(rng, (tokens, 8), "f32")
    got = cuda_lib.embed_bwd(torch.from_numpy(ids).cuda(), dy.cuda(), vocab)
    # the same tokens among 5000: every row the same bits, whichever kernel sorts
    more = np.concatenate([ids, np.full(5000 - tokens, -1)])
    fill = torch.cat([dy, draw(rng, (5000 - tokens, 8), "f32")])
    other = cuda_lib.embed_bwd(torch.from_numpy(more).cuda(), fill.cuda(), vocab)
    assert torch.equal(bits(got), bits(other))
    assert_close(got, embed_bwd(ids, f64(dy), vocab, 1.0), _grad_bound(ids, f64(dy), vocab, 1.0), "dtable")


def test_order_is_the_declared_one(cuda_lib):
    # leaves of 32 tokens summed in token order, joined by the pairwise tree, in
    # fp32 on the host: the same bits
    rng = np.random.default_rng(3)
    tokens, vocab, width = 1500, 5, 24
    ids = rng.choice(vocab, tokens, p=[0.7, 0.2, 0.06, 0.04, 0.0])
    dy = draw(rng, (tokens, width), "f32").numpy()
    got = cuda_lib.embed_bwd(torch.from_numpy(ids).cuda(), torch.from_numpy(dy).cuda(), vocab).cpu().numpy()
    for v in range(vocab):
        rows = dy[ids == v]
        nodes = []
        for l in range(0, len(rows), 32):
            s = np.full(width, -0.0, np.float32)
            for r in rows[l:l + 32]:
                s = s + r
            nodes.append(s)
        while len(nodes) > 1:
            nodes = [nodes[i] + nodes[i + 1] if i + 1 < len(nodes) else nodes[i]
                     for i in range(0, len(nodes), 2)]
        want = nodes[0] if nodes else np.zeros(width, np.float32)
        assert np.array_equal(got[v].view(np.int32), want.view(np.int32)), v


def test_a_row_depends_on_its_own_tokens_only(cuda_lib):
    rng = np.random.default_rng(4)
    width, vocab = 256, 1000
    own = torch.from_numpy(rng.standard_normal((150, width)).astype(np.float32)).bfloat16()

    def batch(others, at):
        ids = np.concatenate([rng.integers(0, vocab, others), np.full(150, 500)])
        ids[:others][ids[:others] == 500] = 501
        dy = torch.cat([torch.randn(others, width).bfloat16(), own])
        order = np.argsort(np.concatenate([rng.random(others), np.sort(rng.random(150) * at)]), kind="stable")
        return cuda_lib.embed_bwd(torch.from_numpy(ids[order]).cuda(), dy[order].contiguous().cuda(), vocab)[500]

    want = batch(0, 1.0)
    for others, at in ((1, 1.0), (77, 0.5), (3000, 1.0)):
        assert torch.equal(bits(batch(others, at)), bits(want))


def test_no_tokens(cuda_lib):
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    dy = torch.zeros(0, 64, device="cuda")
    assert cuda_lib.embed_fwd(ids, torch.ones(3, 64, device="cuda")).shape == (0, 64)
    assert torch.equal(cuda_lib.embed_bwd(ids, dy, 300), torch.zeros(300, 64, device="cuda"))
    old = torch.ones(3, 64, device="cuda")
    assert torch.equal(cuda_lib.embed_bwd(ids, dy, 3, dtable=old, accumulate=True), torch.ones_like(old))


def test_writes_only_its_outputs(cuda_lib):
    rng = np.random.default_rng(5)
    tokens, vocab, width = 333, 41, 40
    n, guard = vocab * width, 64
    raw = torch.full((n + 2 * guard,), 7.0, dtype=torch.float16, device="cuda")
    need = int(cuda_lib.load().embed_bwd_workspace_bytes(tokens, width))
    wraw = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    d = raw[guard:guard + n].view(vocab, width)
    ids = torch.from_numpy(_ids(rng, tokens, vocab, "few")).cuda()
    cuda_lib.embed_bwd(ids, draw(rng, (tokens, width), "f16").cuda(), vocab, dtable=d, ws=wraw[256:256 + need])
    assert bool((raw[:guard] == 7).all()) and bool((raw[guard + n:] == 7).all())
    assert bool((wraw[:256] == 0x5A).all()) and bool((wraw[256 + need:] == 0x5A).all())


def test_captured_and_replayed_with_other_ids(cuda_lib):
    rng = np.random.default_rng(6)
    tokens, vocab, width = 2000, 900, 128
    ids = torch.from_numpy(_ids(rng, tokens, vocab, "few")).cuda()
    other = torch.from_numpy(_ids(rng, tokens, vocab, "uniform")).cuda()
    dy = draw(rng, (tokens, width), "bf16").cuda()
    table = draw(rng, (vocab, width), "bf16").cuda()
    want = [(cuda_lib.embed_fwd(i, table, 3.0), cuda_lib.embed_bwd(i, dy, vocab, 3.0)) for i in (ids, other)]
    buf = ids.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, d = cuda_lib.embed_fwd(buf, table, 3.0), cuda_lib.embed_bwd(buf, dy, vocab, 3.0)
    for k, i in enumerate((ids, other, ids)):
        buf.copy_(i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(want[k % 2][0])) and torch.equal(bits(d), bits(want[k % 2][1]))


def test_two_streams_at_once(cuda_lib):
    rng = np.random.default_rng(8)
    work = []
    for k in range(2):
        ids = torch.from_numpy(_ids(rng, 6000, 5000, "few")).cuda()
        dy = draw(rng, (6000, 512), "bf16").cuda()
        work.append((ids, dy, cuda_lib.embed_bwd(ids, dy, 5000)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        got = []
        for s, (ids, dy, _) in zip(streams, work):
            with torch.cuda.stream(s):
                got.append(cuda_lib.embed_bwd(ids, dy, 5000))
        torch.cuda.synchronize()
        for g, (_, _, want) in zip(got, work):
            assert torch.equal(bits(g), bits(want))


def test_autograd(cuda_lib):
    # the loss is linear in the table: its gradient against the oracle's sums,
    # and against a difference along a random direction (exact but for rounding)
    rng = np.random.default_rng(7)
    ids = torch.from_numpy(rng.integers(0, 20, 50)).cuda()
    table = draw(rng, (20, 16), "f32").cuda().requires_grad_(True)
    dy = draw(rng, (50, 16), "f32")
    (cuda_lib.autograd.embedding(ids, table, 4.0) * dy.cuda()).sum().backward()
    want = embed_bwd(ids.cpu().numpy(), f64(dy), 20, 4.0)
    assert_close(table.grad, want, _grad_bound(ids.cpu().numpy(), f64(dy), 20, 4.0), "grad")
    d = rng.standard_normal((20, 16))
    fwd = lambda t: float((embed_fwd(ids.cpu().numpy(), t, 4.0) * f64(dy)).sum())
    diff = (fwd(f64(table) + d) - fwd(f64(table) - d)) / 2
    assert abs(diff - float((f64(table.grad) * d).sum())) <= 320 * 60 * U32 * 4 * 10
