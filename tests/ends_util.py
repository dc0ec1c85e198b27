"""Helpers of the tests of the layer norm, the embedding and the linear cross
entropy: seeded inputs and the elementwise bound they are held to."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U32 = 2.0 ** -24      # half a step of fp32, relative


def bits(t: torch.Tensor) -> torch.Tensor:
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def draw(rng, shape, dtype, scale=1.0, shift=0.0):
    """A CPU tensor of the stored dtype; its fp64 view is what the reference reads."""
    return torch.from_numpy((rng.standard_normal(shape) * scale + shift).astype(np.float32)).to(
        TORCH[dtype] if isinstance(dtype, str) else dtype)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def assert_close(got: torch.Tensor, want, fp32_error, what, roundings=1):
    """|got - want| <= the roundings of the stored type (each half a step,
    relative to the value, half the subnormal spacing at the bottom) plus the
    fp32 error of the value that was rounded."""
    fi = torch.finfo(got.dtype)
    g, want = f64(got), np.asarray(want, dtype=np.float64)
    fp32_error = np.broadcast_to(np.asarray(fp32_error, dtype=np.float64), want.shape)
    half = fi.eps / 2
    lim = fp32_error + roundings * (half * (np.abs(want) + fp32_error)
                                    + fi.smallest_normal * half)
    err = np.abs(g - want)
    bad = ~(err <= lim)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, err - lim, -np.inf))), want.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {want.size} beyond the bound; worst at "
                             f"{i}: got {g[i]!r}, want {want[i]!r}, bound {lim[i]:.3e}")
