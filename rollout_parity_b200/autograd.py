"""torch.autograd wrappers over the C entry points (the forward saves rstd; the
backward reuses it, so the statistic the gradient sees is the forward's).  The
gradients are computed outside of autograd: the layer norm, the embedding and the
linear cross entropy refuse to be differentiated twice.  As with any function of
torch.autograd, a backward pass is captured into a CUDA graph only while no eager
graph of the same leaves is alive."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import ops


class ZeroCentredRMSNorm(torch.autograd.Function):
    """y = x * rstd * (1 + w); x [rows, width] bf16/fp16/fp32, w fp32 [width]."""

    @staticmethod
    def forward(ctx, x, w, eps=1e-6):
        y, rstd = ops.norm_fwd(x, w, eps)
        ctx.save_for_backward(x, w, rstd)
        ctx.eps = eps
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, rstd = ctx.saved_tensors
        dx, dw = ops.norm_bwd(x, w, dy.contiguous(), rstd, ctx.eps)
        return dx, dw, None


class GatedRMSNorm(torch.autograd.Function):
    """y = x * rstd * w * silu(z); x, z [rows, width] bf16/fp16/fp32, w fp32 [width]."""

    @staticmethod
    def forward(ctx, x, z, w, eps=1e-6):
        y, rstd = ops.gated_norm_fwd(x, z, w, eps)
        ctx.save_for_backward(x, z, w, rstd)
        ctx.eps = eps
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, w, rstd = ctx.saved_tensors
        dx, dz, dw = ops.gated_norm_bwd(x, z, w, dy.contiguous(), rstd, ctx.eps)
        return dx, dz, dw, None


class RMSNorm(torch.autograd.Function):
    """y = x * rstd * (w + weight_offset) * act(z) (the offset added only when
    nonzero); act None/"none" (no z), "silu"/"swish" or "sigmoid"."""

    @staticmethod
    def forward(ctx, x, w, z=None, eps=1e-6, weight_offset=1.0, act=None):
        y, rstd = ops.rmsnorm_fwd(x, w, eps, weight_offset, z, act)
        ctx.save_for_backward(x, w, rstd, *(() if z is None else (z,)))
        ctx.eps, ctx.weight_offset, ctx.act, ctx.gated = eps, weight_offset, act, z is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        saved = ctx.saved_tensors
        x, w, rstd = saved[:3]
        z = saved[3] if ctx.gated else None
        dx, dz, dw = ops.rmsnorm_bwd(x, w, dy.contiguous(), rstd, ctx.eps, ctx.weight_offset, z,
                                     ctx.act)
        return dx, dw, dz, None, None, None


class LayerNorm(torch.autograd.Function):
    """y = (x - mean) * rstd * w + b; x [rows, width] bf16/fp16/fp32, w and b (or
    None) fp32 [width]."""

    @staticmethod
    def forward(ctx, x, w, b=None, eps=1e-5):
        y, mean, rstd = ops.layernorm_fwd(x, w, b, eps)
        ctx.save_for_backward(x, w, mean, rstd)
        ctx.biased = b is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, mean, rstd = ctx.saved_tensors
        dx, dw, db = ops.layernorm_bwd(x, w, dy.contiguous(), mean, rstd, want_db=ctx.biased)
        return dx, dw, db, None


class Embedding(torch.autograd.Function):
    """y[t] = scale * table[ids[t]]; ids [tokens] int64, table [vocab, width]
    bf16/fp16/fp32.  The gradient of the table is dense."""

    @staticmethod
    def forward(ctx, ids, table, scale=1.0):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return ops.embed_fwd(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        return None, ops.embed_bwd(ids, dy.contiguous(), ctx.vocab, ctx.scale), None


class LinearCrossEntropy(torch.autograd.Function):
    """nll[r] = -log softmax(s)[target[r]], s = x w^T (softcap 0) or softcap *
    tanh(x w^T / softcap); x [rows, width], w [vocab, width] bf16/fp16, target
    [rows] int64 (outside [0, vocab): ignored)."""

    @staticmethod
    def forward(ctx, x, w, target, softcap=0.0):
        nll, lse = ops.linear_xent_fwd(x, w, target, softcap)
        ctx.save_for_backward(x, w, target, lse)
        ctx.softcap = softcap
        return nll

    @staticmethod
    @once_differentiable
    def backward(ctx, dnll):
        x, w, target, lse = ctx.saved_tensors
        want_dx, want_dw = ctx.needs_input_grad[:2]
        dx, dw = ops.linear_xent_bwd(x, w, target, lse, dnll.contiguous(), ctx.softcap,
                                     want_dx=want_dx, want_dw=want_dw)
        return dx, dw, None, None


def zero_centred_rms_norm(x, w, eps=1e-6):
    return ZeroCentredRMSNorm.apply(x, w, eps)


def gated_rms_norm(x, z, w, eps=1e-6):
    return GatedRMSNorm.apply(x, z, w, eps)


def rms_norm(x, w, z=None, eps=1e-6, weight_offset=1.0, act=None):
    return RMSNorm.apply(x, w, z, eps, weight_offset, act)


def layer_norm(x, w, b=None, eps=1e-5):
    return LayerNorm.apply(x, w, b, eps)


def embedding(ids, table, scale=1.0):
    return Embedding.apply(ids, table, scale)


def linear_cross_entropy(x, w, target, softcap=0.0):
    return LinearCrossEntropy.apply(x, w, target, softcap)
