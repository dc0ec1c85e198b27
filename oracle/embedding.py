"""The embedding and its gradient in fp64, one token at a time."""
from __future__ import annotations

import numpy as np


def embed_fwd(ids, table, scale=1.0):
    y = np.zeros((len(ids), table.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            y[t] = scale * table[v]
    return y


def embed_bwd(ids, dy, vocab, scale=1.0, old=None):
    """dtable [vocab, width]; ``old`` is what the sums are added to."""
    d = np.zeros((vocab, dy.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < vocab:
            d[v] += dy[t]
    return scale * d if old is None else old + scale * d
