"""Layer norm in fp64, written from the formulas with plain loops over rows:
mean, variance as the mean of squared differences, and the gradients of
sum(y * dy)."""
from __future__ import annotations

import numpy as np


def layernorm_fwd(x, w, b=None, eps=1e-5):
    """(y, mean, rstd) of x [rows, width]; b None means no bias."""
    rows, width = x.shape
    y = np.zeros((rows, width))
    mean, rstd = np.zeros(rows), np.zeros(rows)
    for r in range(rows):
        mean[r] = x[r].sum() / width
        c = x[r] - mean[r]
        rstd[r] = 1.0 / np.sqrt((c * c).sum() / width + eps)
        y[r] = c * rstd[r] * w
        if b is not None:
            y[r] += b
    return y, mean, rstd


def layernorm_bwd(x, w, dy, eps=1e-5, row_mask=None):
    """(dx, dw, db); rows with row_mask[r] == 0 are left out of dw and db."""
    rows, width = x.shape
    _, mean, rstd = layernorm_fwd(x, w, None, eps)
    dx = np.zeros((rows, width))
    dw, db = np.zeros(width), np.zeros(width)
    for r in range(rows):
        xh = (x[r] - mean[r]) * rstd[r]
        g = w * dy[r]
        dx[r] = rstd[r] * (g - g.sum() / width - xh * ((g * xh).sum() / width))
        if row_mask is None or row_mask[r]:
            dw += dy[r] * xh
            db += dy[r]
    return dx, dw, db
