"""Linear cross entropy in fp64: logits, log-sum-exp, the loss of one target per
row and the gradients of sum(dnll * nll), row by row."""
from __future__ import annotations

import numpy as np


def linear_xent(x, w, target, dnll=None, softcap=0.0):
    """(nll, lse) or, with dnll, (nll, lse, dx, dw, |dz|): x [rows, H], w [V, H].
    A target outside [0, V) is ignored: nll 0, no gradient."""
    rows, vocab = x.shape[0], w.shape[0]
    nll, lse = np.zeros(rows), np.zeros(rows)
    dz = np.zeros((rows, vocab))
    for r in range(rows):
        z = w @ x[r]
        t = softcap * np.tanh(z / softcap) if softcap else z
        top = t.max()
        lse[r] = top + np.log(np.exp(t - top).sum())
        if not 0 <= target[r] < vocab:
            continue
        nll[r] = lse[r] - t[target[r]]
        if dnll is not None:
            dz[r] = np.exp(t - lse[r])
            dz[r, target[r]] -= 1.0
            dz[r] *= dnll[r]
            if softcap:
                dz[r] *= 1.0 - (t / softcap) ** 2
    if dnll is None:
        return nll, lse
    kept = (target >= 0) & (target < vocab)
    return nll, lse, dz @ w, dz[kept].T @ x[kept], dz
