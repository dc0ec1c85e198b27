"""The operators together, as a training step of a small language model uses
them: embedding -> layer norm -> gated RMS norm -> layer norm -> linear cross
entropy, with the table tied to the output projection, and the way back."""
import numpy as np
import pytest
import torch

from ends_util import bits, draw

pytestmark = pytest.mark.gpu


def _data(seed, tokens=300, vocab=1000, width=256, dtype=torch.bfloat16):
    rng = np.random.default_rng(seed)
    d = dict(table=draw(rng, (vocab, width), dtype, 0.05), z=draw(rng, (tokens, width), dtype),
             w1=draw(rng, width, "f32", 0.1, 1.0), b1=draw(rng, width, "f32", 0.1),
             w2=draw(rng, width, "f32", 0.1, 1.0), w3=draw(rng, width, "f32", 0.1, 1.0),
             ids=torch.from_numpy(rng.integers(0, vocab, tokens)),
             target=torch.from_numpy(np.where(rng.random(tokens) < 0.3, -100, rng.integers(0, vocab, tokens))))
    return {k: v.cuda() for k, v in d.items()}


def _autograd_step(rn, d, softcap):
    leaves = {k: d[k].clone().requires_grad_(True) for k in ("table", "w1", "b1", "w2", "w3")}
    a = rn.autograd
    h = a.embedding(d["ids"], leaves["table"], 16.0)
    h = a.layer_norm(h, leaves["w1"], leaves["b1"])
    h = a.gated_rms_norm(h, d["z"], leaves["w2"])
    h = a.layer_norm(h, leaves["w3"])
    nll = a.linear_cross_entropy(h, leaves["table"], d["target"], softcap)
    loss = nll.sum() / (d["target"] >= 0).sum()
    loss.backward()
    return nll.detach(), {k: v.grad for k, v in leaves.items()}


def _reference(d, softcap):
    """The same step in fp64 with torch operations."""
    leaves = {k: d[k].double().requires_grad_(True) for k in ("table", "w1", "b1", "w2", "w3")}
    z = d["z"].double()

    def ln(x, w, b=None):
        c = x - x.mean(1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w
        return y if b is None else y + b

    h = ln(leaves["table"][d["ids"]] * 16.0, leaves["w1"], leaves["b1"])
    h = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * leaves["w2"] * z * torch.sigmoid(z)
    h = ln(h, leaves["w3"])
    s = h @ leaves["table"].T
    s = softcap * torch.tanh(s / softcap) if softcap else s
    kept = d["target"] >= 0
    lse = torch.logsumexp(s, 1)
    nll = torch.where(kept, lse - s.gather(1, d["target"].clamp(min=0)[:, None])[:, 0], 0.0)
    (nll.sum() / kept.sum()).backward()
    return nll.detach(), {k: v.grad for k, v in leaves.items()}


@pytest.mark.parametrize("softcap", [0.0, 8.0])
def test_step_against_fp64(cuda_lib, softcap):
    d = _data(0)
    nll, grads = _autograd_step(cuda_lib, d, softcap)
    want_nll, want = _reference(d, softcap)
    # every operator rounds its output to bf16 once (2^-9 rms of the value); five
    # of them forward and five back, the errors adding up at most linearly
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(nll, want_nll) < 5 * 2.0 ** -8
    for k in want:
        assert rel(grads[k], want[k]) < 10 * 2.0 ** -8, (k, rel(grads[k], want[k]))


def test_tied_gradient_by_accumulation(cuda_lib):
    # the head's dW first, the embedding's gradient added to it in place: the
    # same as the sum autograd forms, up to the one rounding it saves
    rn, d = cuda_lib, _data(1)
    h0 = rn.embed_fwd(d["ids"], d["table"], 16.0)
    h1, m1, r1 = rn.layernorm_fwd(h0, d["w1"], d["b1"])
    nll, lse = rn.linear_xent_fwd(h1, d["table"], d["target"])
    g = torch.full_like(nll, 1.0 / 210)
    dh1, dtable = rn.linear_xent_bwd(h1, d["table"], d["target"], lse, g)
    dh0, _, _ = rn.layernorm_bwd(h0, d["w1"], dh1, m1, r1)
    head = dtable.clone()
    rn.embed_bwd(d["ids"], dh0, 1000, 16.0, dtable=dtable, accumulate=True)
    own = rn.embed_bwd(d["ids"], dh0, 1000, 16.0)
    want = head.double() + own.double()
    err = (dtable.double() - want).abs()
    # one rounding of the sum, and the one `own` was rounded with
    assert bool((err <= 2.0 ** -8 * (want.abs() + own.double().abs()) * 1.01 + 1e-30).all())


def test_step_captured_and_replayed(cuda_lib):
    # forward and backward as one graph: other tokens in the same buffers
    rn, d, e = cuda_lib, _data(2), _data(3)
    buf = {k: v.clone() for k, v in d.items()}

    def step(d):
        h0 = rn.embed_fwd(d["ids"], d["table"], 16.0)
        h1, m1, r1 = rn.layernorm_fwd(h0, d["w1"], d["b1"])
        h2, r2 = rn.gated_norm_fwd(h1, d["z"], d["w2"])
        nll, lse = rn.linear_xent_fwd(h2, d["table"], d["target"], 8.0)
        dh2, dtable = rn.linear_xent_bwd(h2, d["table"], d["target"], lse, torch.ones_like(nll), 8.0)
        dh1, dz, dw2 = rn.gated_norm_bwd(h1, d["z"], d["w2"], dh2, r2)
        dh0, dw1, db1 = rn.layernorm_bwd(h0, d["w1"], dh1, m1, r1)
        rn.embed_bwd(d["ids"], dh0, 1000, 16.0, dtable=dtable, accumulate=True)
        return nll, dtable, dz, dw1, db1, dw2

    want = [[t.clone() for t in step(x)] for x in (d, e)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(buf)
    for i, x in enumerate((d, e, d)):
        for k in buf:
            buf[k].copy_(x[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i % 2]):
            assert torch.equal(bits(a), bits(b))


def test_launch_counts(cuda_lib):
    # rn_last_launches counts what the last call enqueued
    rn, d = cuda_lib, _data(4)
    lib = rn.load()
    h0 = rn.embed_fwd(d["ids"], d["table"])
    assert lib.rn_last_launches() == 1
    _, m, r = rn.layernorm_fwd(h0, d["w1"])
    assert lib.rn_last_launches() == 1
    _, lse = rn.linear_xent_fwd(h0, d["table"], d["target"])
    assert lib.rn_last_launches() == 2                       # tiles, join
    rn.linear_xent_bwd(h0, d["table"], d["target"], lse, torch.ones_like(lse))
    assert lib.rn_last_launches() == 4                       # pack, dz, gradients, fold
    rn.layernorm_bwd(h0, d["w1"], h0.clone(), m, r)
    assert lib.rn_last_launches() == 2                       # rows, fold
    rn.embed_bwd(d["ids"], h0, 1000)
    assert lib.rn_last_launches() == 3                       # sort, reduce, join
