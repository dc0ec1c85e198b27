"""The linear cross entropy without a GPU: argument checks (validate-only mode;
the addresses are never dereferenced), workspace sizes, the fp64 formulas."""
import numpy as np
import pytest
import torch

import rollout_parity_b200 as rn
from oracle.xent import linear_xent
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
    return (1 << 44) + (i << 40) + off


X, W, T, NLL, LSE, G, DX, DW, WS = range(9)
R, H, V = 500, 512, 50000


def fwd(lib, rows=R, width=H, vocab=V, dt=DType.BF16, cap=0.0, ws_bytes=None, **kw):
    p = dict(x=P(X), w=P(W), t=P(T), nll=P(NLL), lse=P(LSE), ws=P(WS)) | kw
    n = lib.linear_xent_fwd_workspace_bytes(rows, vocab) if ws_bytes is None else ws_bytes
    return lib.linear_xent_fwd(rows, width, vocab, dt, p["x"], p["w"], p["t"], cap, p["nll"], p["lse"], p["ws"], n, None)


def bwd(lib, rows=R, width=H, vocab=V, dt=DType.BF16, cap=0.0, ws_bytes=None, **kw):
    p = dict(x=P(X), w=P(W), t=P(T), lse=P(LSE), g=P(G), dx=P(DX), dw=P(DW), ws=P(WS)) | kw
    n = lib.linear_xent_bwd_workspace_bytes(rows, width, vocab) if ws_bytes is None else ws_bytes
    return lib.linear_xent_bwd(rows, width, vocab, dt, p["x"], p["w"], p["t"], p["lse"], p["g"], cap, p["dx"], p["dw"],
                               p["ws"], n, None)


COMMON = [
    ({}, Status.OK), (dict(dt=DType.F16, cap=30.0), Status.OK), (dict(rows=1 << 22, vocab=1000), Status.OK),
    (dict(rows=-1), Status.E_ARG), (dict(rows=(1 << 22) + 1), Status.E_ARG), (dict(vocab=0), Status.E_ARG),
    (dict(vocab=(1 << 24) + 1), Status.E_ARG), (dict(cap=-1.0), Status.E_ARG), (dict(cap=float("nan")), Status.E_ARG),
    (dict(cap=2.0 ** -100), Status.OK), (dict(cap=2.0 ** 100), Status.OK), (dict(cap=2.0 ** -101), Status.E_ARG),
    (dict(cap=2.0 ** 101), Status.E_ARG),
    (dict(cap=float("inf")), Status.E_ARG), (dict(dt=DType.F32), Status.E_DTYPE), (dict(dt=9), Status.E_DTYPE),
    (dict(width=100), Status.E_WIDTH), (dict(width=16392), Status.E_WIDTH), (dict(x=0), Status.E_ARG),
    (dict(w=0), Status.E_ARG), (dict(t=0), Status.E_ARG), (dict(x=P(X, 8)), Status.E_ALIGN),
    (dict(w=P(W, 2)), Status.E_ALIGN), (dict(t=P(T, 4)), Status.E_ALIGN), (dict(lse=P(LSE, 2)), Status.E_ALIGN),
    (dict(ws=0), Status.E_WORKSPACE), (dict(ws_bytes=256), Status.E_WORKSPACE), (dict(ws=P(WS, 8)), Status.E_ALIGN),
    (dict(ws=P(W, 64)), Status.E_ARG)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(rows=0, x=0, t=0, nll=0, lse=0, ws=0), Status.OK), (dict(nll=0), Status.OK), (dict(lse=0), Status.OK),
    (dict(nll=0, lse=0), Status.E_ARG), (dict(nll=P(LSE)), Status.E_ARG), (dict(nll=P(T)), Status.E_ARG)])
def test_forward_checks(lib, kw, want):
    assert fwd(lib, **kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(rows=0, x=0, t=0, lse=0, g=0, ws=0), Status.OK), (dict(dx=0), Status.OK), (dict(dw=0), Status.OK),
    (dict(dx=0, dw=0), Status.E_ARG), (dict(lse=0), Status.E_ARG), (dict(g=0), Status.E_ARG),
    (dict(g=P(G, 1)), Status.E_ALIGN), (dict(dx=P(DX, 2)), Status.E_ALIGN), (dict(dx=P(X)), Status.E_ARG),
    (dict(dw=P(W)), Status.E_ARG), (dict(dw=P(DX, 1024)), Status.E_ARG)])
def test_backward_checks(lib, kw, want):
    assert bwd(lib, **kw) == want


def test_workspace_sizes(lib):
    f, b = lib.linear_xent_fwd_workspace_bytes, lib.linear_xent_bwd_workspace_bytes
    assert f(0, V) == 0 and f(5, 0) == 0 and b(0, H, V) == 0 and b(5, 12, V) == 0
    # two floats for every 128 logits (rows rounded up to 256), and a float a row
    assert 512 * 20 * 8 + 512 * 4 <= f(512, 2560) <= 512 * 20 * 8 + 512 * 4 + 256
    # never the logits of the whole vocabulary of a large batch
    assert b(65536, 2048, 151936) < 65536 * 151936 * 2 // 4


def test_binding_refuses_before_the_library():
    x, w, t = torch.zeros(4, 8).half(), torch.zeros(10, 8).half(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        rn.linear_xent_fwd(x, w, t)


@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_formulas_match_differences(cap):
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((4, 6)), rng.standard_normal((9, 6))
    t, g = np.array([2, -1, 8, 0]), rng.standard_normal(4)
    _, _, dx, dw, _ = linear_xent(x, w, t, g, cap)
    loss = lambda x, w: (linear_xent(x, w, t, None, cap)[0] * g).sum()
    for r, k in ((0, 1), (1, 2), (3, 5)):
        e = np.zeros_like(x)
        e[r, k] = 1e-5
        assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-5 - dx[r, k]) < 1e-8
    for v, k in ((2, 1), (5, 0), (0, 4)):
        e = np.zeros_like(w)
        e[v, k] = 1e-5
        assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-5 - dw[v, k]) < 1e-8
