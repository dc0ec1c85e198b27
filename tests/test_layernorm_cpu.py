"""Layer norm without a GPU: the argument checks of the C calls (validate-only
mode; the addresses are never dereferenced) and the fp64 formulas' own check."""
import numpy as np
import pytest

import rollout_parity_b200 as rn
from oracle.layernorm import layernorm_bwd, layernorm_fwd
from rollout_parity_b200 import build as rn_build
from rollout_parity_b200._lib import DType, Status


@pytest.fixture(scope="module")
def lib():
    rn_build.build()
    lib = rn.load()
    lib.rn_test_set_validate_only(1)
    yield lib
    lib.rn_test_set_validate_only(0)


def P(i, off=0):
    return (1 << 40) + (i << 32) + off


X, W, B, Y, M, R, DY, DX, DW, DB, WS, MASK = range(12)
ROWS, H = 640, 1024
TB = ROWS * H * 2


def fwd(lib, rows=ROWS, width=H, eps=1e-5, dt=DType.BF16, **kw):
    p = dict(x=P(X), w=P(W), b=P(B), y=P(Y), mean=P(M), rstd=P(R)) | kw
    return lib.layernorm_fwd(rows, width, eps, dt, p["x"], p["w"], p["b"], p["y"], p["mean"],
                             p["rstd"], None)


def bwd(lib, rows=ROWS, width=H, dt=DType.BF16, ws_bytes=None, **kw):
    p = dict(x=P(X), w=P(W), dy=P(DY), mean=P(M), rstd=P(R), mask=P(MASK), dx=P(DX), dw=P(DW),
             db=P(DB), ws=P(WS)) | kw
    n = lib.layernorm_bwd_workspace_bytes(rows, width, dt) if ws_bytes is None else ws_bytes
    return lib.layernorm_bwd(rows, width, dt, p["x"], p["w"], p["dy"], p["mean"], p["rstd"],
                             p["mask"], p["dx"], p["dw"], p["db"], p["ws"], n, None)


@pytest.mark.parametrize("kw,want", [
    ({}, Status.OK), (dict(b=0, mean=0, rstd=0), Status.OK), (dict(rows=0, x=0, y=0), Status.OK),
    (dict(y=P(X)), Status.OK), (dict(dt=DType.F32), Status.OK),
    (dict(rows=-1), Status.E_ARG), (dict(rows=(1 << 36) + 1), Status.E_ARG),
    (dict(eps=-1.0), Status.E_ARG), (dict(eps=float("nan")), Status.E_ARG),
    (dict(dt=9), Status.E_DTYPE), (dict(width=12), Status.E_WIDTH), (dict(width=16392), Status.E_WIDTH),
    (dict(x=0), Status.E_ARG), (dict(w=0), Status.E_ARG), (dict(y=0), Status.E_ARG),
    (dict(x=P(X, 2)), Status.E_ALIGN), (dict(b=P(B, 4)), Status.E_ALIGN), (dict(mean=P(M, 2)), Status.E_ALIGN),
    (dict(y=P(X, 16)), Status.E_ARG), (dict(y=P(W)), Status.E_ARG), (dict(mean=P(R)), Status.E_ARG),
])
def test_forward_checks(lib, kw, want):
    assert fwd(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({}, Status.OK), (dict(db=0, mask=0), Status.OK), (dict(dx=P(DY)), Status.OK),
    (dict(rows=0, x=0, dy=0, mean=0, rstd=0, dx=0, ws=0), Status.OK),
    (dict(rows=1, ws=0), Status.OK),                       # one block of rows: no workspace
    (dict(rows=-1), Status.E_ARG), (dict(dt=9), Status.E_DTYPE), (dict(width=4), Status.E_WIDTH),
    (dict(dw=0), Status.E_ARG), (dict(mean=0), Status.E_ARG), (dict(rstd=0), Status.E_ARG), (dict(dx=0), Status.E_ARG),
    (dict(dw=P(DW, 4)), Status.E_ALIGN), (dict(db=P(DB, 8)), Status.E_ALIGN), (dict(ws=P(WS, 4)), Status.E_ALIGN),
    (dict(ws=0), Status.E_WORKSPACE), (dict(ws_bytes=15), Status.E_WORKSPACE),
    (dict(dx=P(X)), Status.E_ARG), (dict(dw=P(DB)), Status.E_ARG), (dict(ws=P(X, TB - 16)), Status.E_ARG),
    (dict(dw=P(MASK)), Status.E_ARG),
])
def test_backward_checks(lib, kw, want):
    assert bwd(lib, **kw) == want


def test_workspace_sizes(lib):
    ws = lib.layernorm_bwd_workspace_bytes
    assert ws(0, H, DType.BF16) == 0 and ws(-1, H, DType.BF16) == 0
    assert ws(ROWS, 12, DType.BF16) == 0 and ws(ROWS, H, 9) == 0
    # a bounded number of CTAs writes partials, however many rows
    assert ws(1 << 36, H, DType.BF16) <= 740 * H * 8


def test_formulas_match_differences():
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((3, 16)), rng.standard_normal((3, 16))
    w, b = rng.standard_normal(16), rng.standard_normal(16)
    dx, dw, db = layernorm_bwd(x, w, dy)
    h = 1e-5

    def loss(x, w, b):
        return (layernorm_fwd(x, w, b)[0] * dy).sum()

    for k in range(16):
        e = np.zeros(16)
        e[k] = h
        assert abs((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h) - dw[k]) < 1e-8
        assert abs((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h) - db[k]) < 1e-8
        ex = np.zeros((3, 16))
        ex[1, k] = h
        assert abs((loss(x + ex, w, b) - loss(x - ex, w, b)) / (2 * h) - dx[1, k]) < 1e-8
    assert np.array_equal(layernorm_bwd(x, w, dy, row_mask=np.zeros(3))[1], np.zeros(16))
