"""Python binding of librn, one function per C entry point, same names.

These functions only marshal arguments: they check that torch tensors can be
described by plain pointers (CUDA, contiguous, the right dtype and shape),
allocate outputs the caller did not pass (torch is used for device memory and
streams only), and call the C ABI on the tensors' device and current stream.
Every step of the computation runs in librn's kernels; a failed status raises
RNError.

With ``stream`` the call runs there, but outputs it allocates come from the current
stream's memory: let ``stream`` wait for the current stream before the call, and
the current stream for ``stream`` before an output is used or freed.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._lib import Act, DType, check, load

_DT = {torch.bfloat16: DType.BF16, torch.float16: DType.F16, torch.float32: DType.F32}
# gate activation names; "swish" is another name for silu
_ACT = {None: Act.NONE, "none": Act.NONE, "silu": Act.SILU, "swish": Act.SILU,
        "sigmoid": Act.SIGMOID}


def _dt(x: torch.Tensor) -> DType:
    if x.dtype not in _DT:
        raise TypeError(f"x dtype {x.dtype} not supported (bf16, fp16 or fp32)")
    return _DT[x.dtype]


def act_code(act) -> Act:
    """The C enum for an activation name (None/"none", "silu"/"swish",
    "sigmoid") or an Act value."""
    if isinstance(act, Act):
        return act
    key = act.lower() if isinstance(act, str) else act
    if key not in _ACT:
        raise ValueError(f"unknown activation {act!r} (none, silu, swish or sigmoid)")
    return _ACT[key]


def _mat(name: str, t: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not like.dtype or t.shape != like.shape or t.device != like.device:
        raise ValueError(f"{name} must be {tuple(like.shape)} {like.dtype} on {like.device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _vec(name: str, t: Optional[torch.Tensor], n: int, device) -> torch.Tensor:
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not torch.float32 or t.shape != (n,) or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 [{n}] tensor on {device}")
    return t


def _rows_width(x: torch.Tensor) -> Tuple[int, int]:
    if x.dim() != 2:
        raise ValueError("x must be [rows, width]")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    return int(x.shape[0]), int(x.shape[1])


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(x: torch.Tensor, stream) -> int:
    """The cudaStream_t handle: the tensors' current stream when None, a
    torch.cuda.Stream's handle, or a raw handle passed as an int."""
    if isinstance(stream, int):
        return stream
    s = torch.cuda.current_stream(x.device) if stream is None else stream
    return s.cuda_stream


def _launch(name: str, x: torch.Tensor, stream, *args) -> None:
    """Calls the C entry point ``name`` on x's device (made current only when it
    is not: the context manager costs more than a small call's checks) and on
    ``stream``, or that device's current stream when None."""
    fn = getattr(load(), name)
    index = x.device.index
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(x, stream)
    if index == torch.cuda.current_device():
        status = fn(*args, s)
    else:
        with torch.cuda.device(index):
            status = fn(*args, s)
    check(name, status)


def norm_bwd_workspace_bytes(rows: int, width: int) -> int:
    return int(load().norm_bwd_workspace_bytes(rows, width))


def workspace(rows: int, width: int, device) -> torch.Tensor:
    """A device buffer large enough for the backward's dw partials."""
    n = norm_bwd_workspace_bytes(rows, width)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def rmsnorm_fwd(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, weight_offset: float = 1.0,
                z: Optional[torch.Tensor] = None, act=None, *,
                y: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                want_rstd: bool = True, stream=None):
    """General forward y = x * rstd * (w + weight_offset) * act(z) (the offset
    is added only when nonzero; act None means no gate and no z).  Returns
    (y, rstd)."""
    rows, width = _rows_width(x)
    a = act_code(act)
    if a == Act.NONE:
        if z is not None:
            raise ValueError("z given without a gate activation")
    else:
        _mat("z", z, x)
    _vec("w", w, width, x.device)
    y = torch.empty_like(x) if y is None else _mat("y", y, x)
    if rstd is None and want_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    with torch.cuda.device(x.device):
        check("rmsnorm_fwd",
              load().rmsnorm_fwd(rows, width, eps, weight_offset, int(a), _dt(x), _ptr(x), _ptr(z),
                                 _ptr(w), _ptr(y), _ptr(rstd), _stream(x, stream)))
    return y, rstd


def rmsnorm_add_fwd(x: torch.Tensor, r: torch.Tensor, w: torch.Tensor, eps: float = 1e-6,
                    weight_offset: float = 1.0, z: Optional[torch.Tensor] = None, act=None, *,
                    h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    rstd: Optional[torch.Tensor] = None, want_rstd: bool = True, stream=None):
    """Residual-add forward: h = x + r (rounded once to x's dtype) and the norm
    of h.  Returns (h, y, rstd).  h may be x or r itself (in place)."""
    rows, width = _rows_width(x)
    a = act_code(act)
    _mat("r", r, x)
    if a == Act.NONE:
        if z is not None:
            raise ValueError("z given without a gate activation")
    else:
        _mat("z", z, x)
    _vec("w", w, width, x.device)
    h = torch.empty_like(x) if h is None else _mat("h", h, x)
    y = torch.empty_like(x) if y is None else _mat("y", y, x)
    if rstd is None and want_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    with torch.cuda.device(x.device):
        check("rmsnorm_add_fwd",
              load().rmsnorm_add_fwd(rows, width, eps, weight_offset, int(a), _dt(x), _ptr(x),
                                     _ptr(r), _ptr(z), _ptr(w), _ptr(h), _ptr(y), _ptr(rstd),
                                     _stream(x, stream)))
    return h, y, rstd


def rmsnorm_add_bwd(h: torch.Tensor, w: torch.Tensor, dy: torch.Tensor,
                    dh: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, weight_offset: float = 1.0,
                    z: Optional[torch.Tensor] = None, act=None, *,
                    row_mask: Optional[torch.Tensor] = None,
                    dx: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
                    dw: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None):
    """Residual-add backward: the norm's gradient at h plus dh (the gradient
    of the residual output), the gradient of both x and r.  Returns (dx, dz, dw)."""
    rows, width = _rows_width(h)
    a = act_code(act)
    if a == Act.NONE:
        if z is not None or dz is not None:
            raise ValueError("z or dz given without a gate activation")
    else:
        _mat("z", z, h)
        dz = torch.empty_like(h) if dz is None else _mat("dz", dz, h)
    _vec("w", w, width, h.device)
    _mat("dy", dy, h)
    if dh is not None:
        _mat("dh", dh, h)
    if rstd is not None:
        _vec("rstd", rstd, rows, h.device)
    if row_mask is not None:
        if row_mask.dtype not in (torch.bool, torch.uint8) or tuple(row_mask.shape) != (rows,) \
                or row_mask.device != h.device or not row_mask.is_contiguous():
            raise ValueError(f"row_mask must be a contiguous bool/uint8 [{rows}] tensor on {h.device}")
        row_mask = row_mask.view(torch.uint8)
    dx = torch.empty_like(h) if dx is None else _mat("dx", dx, h)
    dw = torch.empty(width, dtype=torch.float32, device=h.device) if dw is None else \
        _vec("dw", dw, width, h.device)
    ws, nws = _ws(rows, width, h.device, ws)
    with torch.cuda.device(h.device):
        check("rmsnorm_add_bwd",
              load().rmsnorm_add_bwd(rows, width, eps, weight_offset, int(a), _dt(h), _ptr(h),
                                     _ptr(z), _ptr(w), _ptr(dy), _ptr(dh), _ptr(rstd),
                                     _ptr(row_mask), _ptr(dx), _ptr(dz), _ptr(dw), _ptr(ws), nws,
                                     _stream(h, stream)))
    return dx, dz, dw


def norm_fwd(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, *,
             y: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
             want_rstd: bool = True, stream=None):
    """Zero-centred RMSNorm forward.  Returns (y, rstd); rstd is None when
    want_rstd is False and none was passed."""
    rows, width = _rows_width(x)
    _vec("w", w, width, x.device)
    y = torch.empty_like(x) if y is None else _mat("y", y, x)
    if rstd is None and want_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    with torch.cuda.device(x.device):
        check("norm_fwd", load().norm_fwd(rows, width, eps, _dt(x), _ptr(x), _ptr(w), _ptr(y),
                                          _ptr(rstd), _stream(x, stream)))
    return y, rstd


def gated_norm_fwd(x: torch.Tensor, z: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, *,
                   y: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                   want_rstd: bool = True, stream=None):
    """Gated RMSNorm forward.  Returns (y, rstd)."""
    rows, width = _rows_width(x)
    _mat("z", z, x)
    _vec("w", w, width, x.device)
    y = torch.empty_like(x) if y is None else _mat("y", y, x)
    if rstd is None and want_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    with torch.cuda.device(x.device):
        check("gated_norm_fwd",
              load().gated_norm_fwd(rows, width, eps, _dt(x), _ptr(x), _ptr(z), _ptr(w), _ptr(y),
                                    _ptr(rstd), _stream(x, stream)))
    return y, rstd


def _ws(rows, width, device, ws):
    if ws is None:
        ws = workspace(rows, width, device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous buffer on the tensors' device")
    return ws, ws.numel() * ws.element_size()


def rmsnorm_bwd(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor,
                rstd: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_offset: float = 1.0,
                z: Optional[torch.Tensor] = None, act=None, *,
                row_mask: Optional[torch.Tensor] = None,
                dx: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
                dw: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream=None):
    """General backward.  Returns (dx, dz, dw); dz is None without a gate.
    rstd=None recomputes it.  row_mask ([rows] bool or uint8): rows where it is
    zero are left out of dw (dx and dz are still every row's)."""
    rows, width = _rows_width(x)
    a = act_code(act)
    if a == Act.NONE:
        if z is not None or dz is not None:
            raise ValueError("z or dz given without a gate activation")
    else:
        _mat("z", z, x)
        dz = torch.empty_like(x) if dz is None else _mat("dz", dz, x)
    _vec("w", w, width, x.device)
    _mat("dy", dy, x)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    if row_mask is not None:
        if row_mask.dtype not in (torch.bool, torch.uint8) or tuple(row_mask.shape) != (rows,) \
                or row_mask.device != x.device or not row_mask.is_contiguous():
            raise ValueError(f"row_mask must be a contiguous bool/uint8 [{rows}] tensor on {x.device}")
        row_mask = row_mask.view(torch.uint8)
    dx = torch.empty_like(x) if dx is None else _mat("dx", dx, x)
    dw = torch.empty(width, dtype=torch.float32, device=x.device) if dw is None else \
        _vec("dw", dw, width, x.device)
    ws, nws = _ws(rows, width, x.device, ws)
    with torch.cuda.device(x.device):
        check("rmsnorm_bwd",
              load().rmsnorm_bwd(rows, width, eps, weight_offset, int(a), _dt(x), _ptr(x), _ptr(z),
                                 _ptr(w), _ptr(dy), _ptr(rstd), _ptr(row_mask), _ptr(dx),
                                 _ptr(dz), _ptr(dw), _ptr(ws), nws, _stream(x, stream)))
    return dx, dz, dw


def norm_bwd(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor,
             rstd: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
             dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None, stream=None):
    """Zero-centred RMSNorm backward.  Returns (dx, dw).  rstd=None recomputes it."""
    rows, width = _rows_width(x)
    _vec("w", w, width, x.device)
    _mat("dy", dy, x)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    dx = torch.empty_like(x) if dx is None else _mat("dx", dx, x)
    dw = torch.empty(width, dtype=torch.float32, device=x.device) if dw is None else \
        _vec("dw", dw, width, x.device)
    ws, nws = _ws(rows, width, x.device, ws)
    with torch.cuda.device(x.device):
        check("norm_bwd", load().norm_bwd(rows, width, eps, _dt(x), _ptr(x), _ptr(w), _ptr(dy),
                                          _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(ws), nws,
                                          _stream(x, stream)))
    return dx, dw


def gated_norm_bwd(x: torch.Tensor, z: torch.Tensor, w: torch.Tensor, dy: torch.Tensor,
                   rstd: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                   dx: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
                   dw: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                   stream=None):
    """Gated RMSNorm backward.  Returns (dx, dz, dw).  rstd=None recomputes it."""
    rows, width = _rows_width(x)
    _mat("z", z, x)
    _vec("w", w, width, x.device)
    _mat("dy", dy, x)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    dx = torch.empty_like(x) if dx is None else _mat("dx", dx, x)
    dz = torch.empty_like(x) if dz is None else _mat("dz", dz, x)
    dw = torch.empty(width, dtype=torch.float32, device=x.device) if dw is None else \
        _vec("dw", dw, width, x.device)
    ws, nws = _ws(rows, width, x.device, ws)
    with torch.cuda.device(x.device):
        check("gated_norm_bwd",
              load().gated_norm_bwd(rows, width, eps, _dt(x), _ptr(x), _ptr(z), _ptr(w), _ptr(dy),
                                    _ptr(rstd), _ptr(dx), _ptr(dz), _ptr(dw), _ptr(ws), nws,
                                    _stream(x, stream)))
    return dx, dz, dw


def rmsnorm_bwd_chunks(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor,
                       rstd: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       weight_offset: float = 1.0, z: Optional[torch.Tensor] = None, act=None, *,
                       row_mask: Optional[torch.Tensor] = None,
                       dx: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
                       dw_chunks: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, stream=None):
    """rmsnorm_bwd returning dw's 256-row chunk partials [ceil(rows/256), width]
    in place of dw (for the data-parallel fold).  Returns (dx, dz, dw_chunks)."""
    rows, width = _rows_width(x)
    a = act_code(act)
    if a == Act.NONE:
        if z is not None or dz is not None:
            raise ValueError("z or dz given without a gate activation")
    else:
        _mat("z", z, x)
        dz = torch.empty_like(x) if dz is None else _mat("dz", dz, x)
    _vec("w", w, width, x.device)
    _mat("dy", dy, x)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    if row_mask is not None:
        if row_mask.dtype not in (torch.bool, torch.uint8) or tuple(row_mask.shape) != (rows,) \
                or row_mask.device != x.device or not row_mask.is_contiguous():
            raise ValueError(f"row_mask must be a contiguous bool/uint8 [{rows}] tensor on {x.device}")
        row_mask = row_mask.view(torch.uint8)
    nc = int(load().rmsnorm_bwd_chunk_count(rows))
    dx = torch.empty_like(x) if dx is None else _mat("dx", dx, x)
    if dw_chunks is None:
        dw_chunks = torch.empty(nc, width, dtype=torch.float32, device=x.device)
    elif (dw_chunks.device != x.device or dw_chunks.dtype != torch.float32
          or tuple(dw_chunks.shape) != (nc, width) or not dw_chunks.is_contiguous()):
        raise ValueError(f"dw_chunks must be a contiguous fp32 [{nc}, {width}] tensor on {x.device}")
    ws, nws = _ws(rows, width, x.device, ws)
    with torch.cuda.device(x.device):
        check("rmsnorm_bwd_chunks",
              load().rmsnorm_bwd_chunks(rows, width, eps, weight_offset, int(a), _dt(x), _ptr(x),
                                        _ptr(z), _ptr(w), _ptr(dy), _ptr(rstd), _ptr(row_mask),
                                        _ptr(dx), _ptr(dz), _ptr(dw_chunks), _ptr(ws), nws,
                                        _stream(x, stream)))
    return dx, dz, dw_chunks


def rn_fold_tree(partials: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The level-by-level pairwise tree over the rows of a [n, width] fp32 CUDA
    tensor (any n >= 1); returns the [width] result."""
    if partials.dim() != 2 or partials.dtype != torch.float32 or not partials.is_cuda \
            or not partials.is_contiguous():
        raise ValueError("partials must be a contiguous fp32 CUDA tensor [n, width]")
    n, width = int(partials.shape[0]), int(partials.shape[1])
    out = torch.empty(width, dtype=torch.float32, device=partials.device) if out is None else \
        _vec("out", out, width, partials.device)
    if ws is None:
        nb = int(load().rn_fold_tree_workspace_bytes(n, width))
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=partials.device)
    with torch.cuda.device(partials.device):
        check("rn_fold_tree", load().rn_fold_tree(n, width, _ptr(partials), _ptr(out), _ptr(ws),
                                                  ws.numel() * ws.element_size(),
                                                  _stream(partials, stream)))
    return out


def rn_fold_rows(partials: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Joins the rows of a [n, width] fp32 CUDA tensor of dw partials with the
    backward's pairwise tree; returns the [width] result."""
    if partials.dim() != 2 or partials.dtype != torch.float32 or not partials.is_cuda \
            or not partials.is_contiguous():
        raise ValueError("partials must be a contiguous fp32 CUDA tensor [n, width]")
    n, width = int(partials.shape[0]), int(partials.shape[1])
    out = torch.empty(width, dtype=torch.float32, device=partials.device) if out is None else \
        _vec("out", out, width, partials.device)
    with torch.cuda.device(partials.device):
        check("rn_fold_rows", load().rn_fold_rows(n, width, _ptr(partials), _ptr(out),
                                                  _stream(partials, stream)))
    return out


def _row_mask(row_mask: Optional[torch.Tensor], rows: int, device) -> Optional[torch.Tensor]:
    if row_mask is None:
        return None
    if row_mask.dtype not in (torch.bool, torch.uint8) or tuple(row_mask.shape) != (rows,) \
            or row_mask.device != device or not row_mask.is_contiguous():
        raise ValueError(f"row_mask must be a contiguous bool/uint8 [{rows}] tensor on {device}")
    return row_mask.view(torch.uint8)


def _buffer(ws: Optional[torch.Tensor], need: int, device,
            stream) -> Tuple[Optional[torch.Tensor], int]:
    """A workspace of at least ``need`` bytes (the caller's is passed through;
    none when none is needed).  It is allocated on the stream that uses it, so
    that the caching allocator does not give it to another stream's work while
    the call still runs."""
    if ws is None:
        if not need:
            return None, 0
        if stream is None:
            return torch.empty(need, dtype=torch.uint8, device=device), need
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device) if stream else \
                torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=device), need
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous buffer on the tensors' device")
    return ws, ws.numel() * ws.element_size()


def layernorm_fwd(x: torch.Tensor, w: torch.Tensor, b: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, *, y: Optional[torch.Tensor] = None,
                  mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                  want_stats: bool = True, stream=None):
    """Layer norm forward y = (x - mean) * rstd * w + b (b None: no bias).
    Returns (y, mean, rstd); the statistics are None when want_stats is False
    and none were passed.  y may be x itself."""
    rows, width = _rows_width(x)
    dt = _dt(x)
    _vec("w", w, width, x.device)
    if b is not None:
        _vec("b", b, width, x.device)
    y = torch.empty_like(x) if y is None else _mat("y", y, x)
    if mean is not None:
        _vec("mean", mean, rows, x.device)
    elif want_stats:
        mean = w.new_empty(rows)
    if rstd is not None:
        _vec("rstd", rstd, rows, x.device)
    elif want_stats:
        rstd = w.new_empty(rows)
    _launch("layernorm_fwd", x, stream, rows, width, eps, dt, _ptr(x), _ptr(w), _ptr(b), _ptr(y),
            _ptr(mean), _ptr(rstd))
    return y, mean, rstd


def layernorm_bwd(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor,
                  rstd: torch.Tensor, *, row_mask: Optional[torch.Tensor] = None,
                  want_db: bool = True, dx: Optional[torch.Tensor] = None,
                  dw: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None, stream=None):
    """Layer norm backward.  Returns (dx, dw, db); db is None when want_db is
    False and none was passed.  row_mask ([rows] bool or uint8): rows where it
    is zero are left out of dw and db.  dx may be dy itself."""
    rows, width = _rows_width(x)
    dt = _dt(x)
    _vec("w", w, width, x.device)
    _mat("dy", dy, x)
    _vec("mean", mean, rows, x.device)
    _vec("rstd", rstd, rows, x.device)
    row_mask = _row_mask(row_mask, rows, x.device)
    dx = torch.empty_like(x) if dx is None else _mat("dx", dx, x)
    dw = torch.empty_like(w) if dw is None else _vec("dw", dw, width, x.device)
    if db is not None:
        _vec("db", db, width, x.device)
    elif want_db:
        db = torch.empty_like(w)
    lib = load()
    ws, nws = _buffer(ws, int(lib.layernorm_bwd_workspace_bytes(rows, width, dt)), x.device,
                      stream)
    _launch("layernorm_bwd", x, stream, rows, width, dt, _ptr(x), _ptr(w), _ptr(dy), _ptr(mean),
            _ptr(rstd), _ptr(row_mask), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), nws)
    return dx, dw, db


def _index(name: str, t: torch.Tensor, device) -> int:
    """The length of an int64 index vector on ``device``."""
    if t.dim() != 1 or t.dtype != torch.int64 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int64 [tokens] tensor on {device}")
    return int(t.shape[0])


def embed_fwd(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, *,
              y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = scale * table[ids[t]], rounded once; table [vocab, width], ids
    [tokens] int64.  An id outside [0, vocab) gives a zero row."""
    vocab, width = _rows_width(table)
    dt = _dt(table)
    tokens = _index("ids", ids, table.device)
    if y is None:
        y = torch.empty(tokens, width, dtype=table.dtype, device=table.device)
    elif y.dtype != table.dtype or y.device != table.device or tuple(y.shape) != (tokens, width) \
            or not y.is_contiguous():
        raise ValueError(f"y must be a contiguous {table.dtype} [{tokens}, {width}] tensor on "
                         f"{table.device}")
    _launch("embed_fwd", table, stream, tokens, vocab, width, scale, dt, _ptr(ids), _ptr(table),
            _ptr(y))
    return y


def embed_bwd(ids: torch.Tensor, dy: torch.Tensor, vocab: int, scale: float = 1.0, *,
              dtable: Optional[torch.Tensor] = None, accumulate: bool = False,
              ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of embed_fwd's table: dtable[v] = scale * the sum of dy[t]
    over the tokens with ids[t] == v, [vocab, width] of dy's dtype.  With
    accumulate, the sums are added to the given dtable."""
    tokens, width = _rows_width(dy)
    dt = _dt(dy)
    if _index("ids", ids, dy.device) != tokens:
        raise ValueError(f"ids must have dy's {tokens} tokens, got {ids.shape[0]}")
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs a dtable to add to")
        dtable = torch.empty(vocab, width, dtype=dy.dtype, device=dy.device)
    elif dtable.dtype != dy.dtype or dtable.device != dy.device \
            or tuple(dtable.shape) != (vocab, width) or not dtable.is_contiguous():
        raise ValueError(f"dtable must be a contiguous {dy.dtype} [{vocab}, {width}] tensor on "
                         f"{dy.device}")
    lib = load()
    ws, nws = _buffer(ws, int(lib.embed_bwd_workspace_bytes(tokens, width)), dy.device,
                      stream)
    _launch("embed_bwd", dy, stream, tokens, vocab, width, scale, dt, _ptr(ids), _ptr(dy),
            int(accumulate), _ptr(dtable), _ptr(ws), nws)
    return dtable


def _head(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor) -> Tuple[int, int, int]:
    """(rows, width, vocab) of a projection x [rows, width] onto w [vocab, width]."""
    rows, width = _rows_width(x)
    if w.dim() != 2 or w.dtype != x.dtype or w.device != x.device or int(w.shape[1]) != width \
            or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous {x.dtype} [vocab, {width}] tensor on {x.device}")
    if _index("target", target, x.device) != rows:
        raise ValueError(f"target must have x's {rows} rows, got {target.shape[0]}")
    return rows, width, int(w.shape[0])


def linear_xent_fwd(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, softcap: float = 0.0, *,
                    nll: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    """The negative log-probability of one target token per row under the
    softmax of x w^T (with softcap > 0, of softcap * tanh(x w^T / softcap)),
    and the log of the softmax's sum.  x [rows, width] and w [vocab, width]
    bf16 or fp16, target [rows] int64 (outside [0, vocab): ignored, nll 0).
    Returns (nll, lse), fp32 [rows]."""
    rows, width, vocab = _head(x, w, target)
    dt = _dt(x)
    nll = torch.empty(rows, dtype=torch.float32, device=x.device) if nll is None else \
        _vec("nll", nll, rows, x.device)
    lse = torch.empty(rows, dtype=torch.float32, device=x.device) if lse is None else \
        _vec("lse", lse, rows, x.device)
    lib = load()
    ws, nws = _buffer(ws, int(lib.linear_xent_fwd_workspace_bytes(rows, vocab)), x.device,
                      stream)
    _launch("linear_xent_fwd", x, stream, rows, width, vocab, dt, _ptr(x), _ptr(w), _ptr(target),
            softcap, _ptr(nll), _ptr(lse), _ptr(ws), nws)
    return nll, lse


def linear_xent_bwd(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                    dnll: torch.Tensor, softcap: float = 0.0, *, want_dx: bool = True,
                    want_dw: bool = True, dx: Optional[torch.Tensor] = None,
                    dw: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None):
    """The gradient of sum(dnll * nll) of linear_xent_fwd (lse from that call).
    Returns (dx, dw) of x's dtype, None for the one not wanted."""
    rows, width, vocab = _head(x, w, target)
    dt = _dt(x)
    _vec("lse", lse, rows, x.device)
    _vec("dnll", dnll, rows, x.device)
    if dx is not None:
        _mat("dx", dx, x)
    elif want_dx:
        dx = torch.empty_like(x)
    if dw is not None:
        _mat("dw", dw, w)
    elif want_dw:
        dw = torch.empty_like(w)
    lib = load()
    ws, nws = _buffer(ws, int(lib.linear_xent_bwd_workspace_bytes(rows, width, vocab)), x.device,
                      stream)
    _launch("linear_xent_bwd", x, stream, rows, width, vocab, dt, _ptr(x), _ptr(w), _ptr(target),
            _ptr(lse), _ptr(dnll), softcap, _ptr(dx), _ptr(dw), _ptr(ws), nws)
    return dx, dw


def rn_describe(width: int, dtype=torch.bfloat16) -> str:
    """The provenance string for (width, dtype): kernels, team shape, reduction
    order, dw tree, accumulator; "unsupported" for an invalid pair."""
    if isinstance(dtype, torch.dtype):
        if dtype not in _DT:
            return "unsupported"
        dt = _DT[dtype]
    else:
        dt = int(dtype)
    return load().rn_describe(width, dt).decode()


def rn_test_set_geometry(max_ctas: int = 0, leaves_per_cta: int = 0, fold_rows: int = 0) -> None:
    check("rn_test_set_geometry", load().rn_test_set_geometry(max_ctas, leaves_per_cta, fold_rows))


def rn_test_set_wait_failed(on: bool) -> None:
    check("rn_test_set_wait_failed", load().rn_test_set_wait_failed(1 if on else 0))


def rn_test_set_validate_only(on: bool) -> None:
    load().rn_test_set_validate_only(1 if on else 0)
