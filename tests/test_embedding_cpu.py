"""The embedding's argument checks without a GPU (validate-only mode; the
addresses are never dereferenced) and the binding's own refusals."""
import pytest
import torch

import rollout_parity_b200 as rn
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
    return (1 << 44) + (i << 40) + off   # 1 TiB apart: the largest table is smaller


IDS, T, Y, DY, D, WS = range(6)
N, V, H = 1000, 50000, 512


def fwd(lib, tokens=N, vocab=V, width=H, scale=1.0, dt=DType.BF16, **kw):
    p = dict(ids=P(IDS), table=P(T), y=P(Y)) | kw
    return lib.embed_fwd(tokens, vocab, width, scale, dt, p["ids"], p["table"], p["y"], None)


def bwd(lib, tokens=N, vocab=V, width=H, scale=1.0, dt=DType.BF16, add=0, ws_bytes=None, **kw):
    p = dict(ids=P(IDS), dy=P(DY), d=P(D), ws=P(WS)) | kw
    n = lib.embed_bwd_workspace_bytes(tokens, width) if ws_bytes is None else ws_bytes
    return lib.embed_bwd(tokens, vocab, width, scale, dt, p["ids"], p["dy"], add, p["d"], p["ws"], n, None)


@pytest.mark.parametrize("kw,want", [
    ({}, Status.OK), (dict(tokens=0, ids=0, y=0), Status.OK), (dict(vocab=1 << 27), Status.OK),
    (dict(tokens=-1), Status.E_ARG), (dict(tokens=(1 << 28) + 1), Status.E_ARG),
    (dict(vocab=0), Status.E_ARG), (dict(vocab=(1 << 27) + 1), Status.E_ARG),
    (dict(scale=float("inf")), Status.E_ARG), (dict(scale=float("nan")), Status.E_ARG),
    (dict(dt=3), Status.E_DTYPE), (dict(width=20), Status.E_WIDTH), (dict(ids=0), Status.E_ARG),
    (dict(table=0), Status.E_ARG), (dict(y=0), Status.E_ARG), (dict(ids=P(IDS, 4)), Status.E_ALIGN),
    (dict(table=P(T, 2)), Status.E_ALIGN), (dict(y=P(Y, 8)), Status.E_ALIGN),
    (dict(y=P(T, V * H * 2 - 16)), Status.E_ARG), (dict(y=P(IDS)), Status.E_ARG)])
def test_forward_checks(lib, kw, want):
    assert fwd(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({}, Status.OK), (dict(add=1), Status.OK), (dict(tokens=0, ids=0, dy=0), Status.OK),
    (dict(tokens=-1), Status.E_ARG), (dict(vocab=0), Status.E_ARG), (dict(scale=float("nan")), Status.E_ARG),
    (dict(dt=3), Status.E_DTYPE), (dict(width=4), Status.E_WIDTH), (dict(dy=0), Status.E_ARG),
    (dict(d=0), Status.E_ARG), (dict(ws=0), Status.E_WORKSPACE), (dict(ws_bytes=100), Status.E_WORKSPACE),
    (dict(ws=P(WS, 8)), Status.E_ALIGN), (dict(d=P(D, 2)), Status.E_ALIGN),
    (dict(d=P(DY, 16)), Status.E_ARG), (dict(ws=P(D, 32)), Status.E_ARG), (dict(d=P(IDS)), Status.E_ARG)])
def test_backward_checks(lib, kw, want):
    assert bwd(lib, **kw) == want


def test_workspace_sizes(lib):
    ws = lib.embed_bwd_workspace_bytes
    assert ws(-1, H) == 0 and ws((1 << 28) + 1, H) == 0 and ws(5, 12) == 0
    assert ws(0, H) > 0
    # 16 bytes a token and two fp32 rows for every 32 tokens, rounded up
    n = 1 << 20
    assert 16 * n + n // 16 * H * 4 <= ws(n, H) <= 17 * n + (n // 16 + 2) * H * 4 + 4096


def test_binding_refuses_before_the_library():
    ids, dy = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        rn.embed_fwd(ids, torch.zeros(10, 8))
    with pytest.raises(ValueError, match="CUDA"):
        rn.embed_bwd(ids, dy, 10)
