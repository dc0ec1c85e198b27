"""The autograd functions of the layer norm, the embedding and the linear cross
entropy without a GPU: what they do with a second derivative.  The operators are
replaced by torch operations that record nothing, as the library's calls do."""
import pytest
import torch

from rollout_parity_b200 import autograd, ops


@pytest.fixture
def plain_ops(monkeypatch):
    def no_grad(f):
        return lambda *a, **k: torch.no_grad()(f)(*a, **k)

    def ln_fwd(x, w, b=None, eps=1e-5):
        var, mean = torch.var_mean(x, 1, correction=0)
        r = torch.rsqrt(var + eps)
        y = (x - mean[:, None]) * r[:, None] * w
        return y if b is None else y + b, mean, r

    def ln_bwd(x, w, dy, mean, rstd, want_db=True):
        return dy * w * rstd[:, None], (dy * x).sum(0), dy.sum(0) if want_db else None

    def embed_bwd(ids, dy, vocab, scale=1.0):
        return torch.zeros(vocab, dy.shape[1]).index_add_(0, ids, dy) * scale

    def xent_fwd(x, w, target, softcap=0.0):
        z = x @ w.T
        lse = torch.logsumexp(z, 1)
        return lse - z.gather(1, target[:, None])[:, 0], lse

    def xent_bwd(x, w, target, lse, dnll, softcap=0.0, want_dx=True, want_dw=True):
        d = torch.exp(x @ w.T - lse[:, None])
        d[torch.arange(len(target)), target] -= 1.0
        d = d * dnll[:, None]
        return d @ w if want_dx else None, d.T @ x if want_dw else None

    for name, f in dict(layernorm_fwd=ln_fwd, layernorm_bwd=ln_bwd, embed_bwd=embed_bwd, linear_xent_fwd=xent_fwd,
                        embed_fwd=lambda ids, table, scale=1.0: table[ids] * scale, linear_xent_bwd=xent_bwd).items():
        monkeypatch.setattr(ops, name, no_grad(f))


def _layer_norm(leaf):
    return autograd.layer_norm(leaf, torch.ones(6), torch.zeros(6))


def _embedding(leaf):
    return autograd.embedding(torch.tensor([1, 0, 3]), leaf, 2.0) ** 2


def _cross_entropy(leaf):
    return autograd.linear_cross_entropy(leaf, torch.eye(6), torch.tensor([1, 0, 3, 5]))


@pytest.mark.parametrize("f", [_layer_norm, _embedding, _cross_entropy])
def test_second_derivatives_are_refused(plain_ops, f):
    # (a first derivative that another is to follow is given; the second is not
    # taken for zero beside a term that has one)
    leaf = torch.randn(4, 6, requires_grad=True)
    first, = torch.autograd.grad((f(leaf) ** 2).sum(), leaf, create_graph=True)
    assert first.shape == leaf.shape
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (first.sum() + (leaf ** 2).sum()).backward()
