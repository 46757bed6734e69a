"""Binding of what stands around the recurrence in a layer: the norm with the residual's
addition, rows in 8-bit integers and their products, and the short convolution for packed
requests.  As in the package's other calls, arguments are checked and marshalled here and
every operation runs in the HIP kernels of ``libselscan.so`` (see ``include/selscan.h``)."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _DTYPES, _at, _check, _dense_like, _lib, _nseq, _rows, _scratch, _stream_at

__all__ = ["rms_bwd_workspace_size", "sscan_rms_fwd", "sscan_rms_bwd", "sscan_i8_quant", "sscan_i8_matmul",
           "dwconv_bwd_workspace_size", "sscan_dwconv_fwd", "sscan_dwconv_bwd", "sscan_dwconv_step"]

_P, _I64, _SZ, _F, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float, ctypes.c_int
for _name, _args, _res in (
        ("sscan_rms_fwd", [_I64] * 2 + [_I] * 2 + [_P, _I64, _P, _P, _F, _P, _P, _P, _I64, _P, _P], _I),
        ("sscan_rms_bwd_workspace_size", [_I64] * 2, _SZ),
        ("sscan_rms_bwd", [_I64] * 2 + [_I] * 2 + [_P, _I64, _P, _F, _P, _P, _P, _I64, _P, _P, _P, _SZ, _P], _I),
        ("sscan_i8_quant", [_I64] * 2 + [_I, _P, _I64, _P, _I64, _P, _P], _I),
        ("sscan_i8_matmul", [_I64] * 3 + [_P, _I64, _P, _P, _I64, _P, _P, _I, _P, _I64, _P], _I),
        ("sscan_dwconv_fwd", [_I64] * 4 + [_I] * 2 + [_P, _I64] + [_P] * 4 + [_I64] + [_P] * 3, _I),
        ("sscan_dwconv_bwd_workspace_size", [_I64] * 4, _SZ),
        ("sscan_dwconv_bwd", [_I64] * 4 + [_I] * 2 + [_P, _I64] + [_P] * 4 + [_I64] + [_P] * 3 + [_I64] + [_P] * 4
         + [_SZ, _P], _I),
        ("sscan_dwconv_step", [_I64] * 3 + [_I] * 2 + [_P, _I64, _P, _P, _P, _I64] + [_P] * 4, _I)):
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _res

_F32, _I8 = torch.float32, torch.int8


def _run(t: torch.Tensor, fn, *args):
    """The call on t's device, on that device's current stream."""
    dev = t.get_device()
    if dev == torch.cuda.current_device():
        rc = fn(*args, _stream_at(t))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream_at(t))
    if rc:
        _check(rc)


def _together(t: torch.Tensor, *others):
    """All tensors of a call are on one device: t's."""
    dev = t.get_device()
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError(f"all tensors must be on one device, got {t.device} and {o.device}")


def _tokens(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """(rows, channels) of a tensor of tokens, [rows, dim] or [batch, seqlen, dim]."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [rows, dim] or [batch, seqlen, dim]")
    return (t.shape[0] if t.dim() == 2 else t.shape[0] * t.shape[1]), t.shape[-1]


def _float(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return _DTYPES[t.dtype]


def _new(x: torch.Tensor, dtype, given: Optional[torch.Tensor], name: str):
    """(dense tensor of x's shape, its address): the given one, checked, or a new one."""
    if given is not None:
        return given, _at(given, name, dtype, x.shape)
    t = torch.empty_like(x, dtype=dtype) if x.is_contiguous() else torch.empty(x.shape, dtype=dtype, device=x.device)
    return t, t.data_ptr()


def _codes(x: torch.Tensor, given: Optional[torch.Tensor]):
    """(codes for x, address, row stride), new ones with rows that start at multiples of 16
    bytes (which sscan_i8_matmul reads fastest)."""
    dim = x.shape[-1]
    if given is not None:
        return (given, *_rows(given, "codes", _I8, x.shape))
    if dim % 16 == 0:
        return (*_new(x, _I8, None, "codes"), dim)
    wide = (dim + 15) // 16 * 16
    t = torch.empty((*x.shape[:-1], wide), dtype=_I8, device=x.device)
    return t[..., :dim], t.data_ptr(), wide


def _scales(x: torch.Tensor, given: Optional[torch.Tensor]):
    """(a scale for each row of x, address)."""
    shape = x.shape[:-1]
    if given is not None:
        return given, _at(given, "scales", _F32, shape)
    t = x.new_empty(shape[0] if len(shape) == 1 else shape, dtype=_F32)      # an int is the cheaper argument
    return t, t.data_ptr()


def rms_bwd_workspace_size(rows: int, dim: int) -> int:
    return int(_lib.sscan_rms_bwd_workspace_size(rows, dim))


def sscan_rms_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, want_y: bool = True, want_codes: bool = False, want_residual: Optional[bool] = None,
                  residual_dtype: Optional[torch.dtype] = None, out: Optional[dict] = None) -> dict:
    """Root-mean-square norm with the residual's addition: s = x + residual, rounded to the
    residual's type; y = s / sqrt(mean(s^2) + eps) * weight.

    x: [rows, dim] or [batch, seqlen, dim] (float32 or bfloat16, dense or columns of a wider
    tensor); residual: x's shape, dense, float32 or x's type; weight [dim] float32 (default
    ones).  Returns a dict with y (want_y), codes and scales (want_codes: y in 8 bits as
    ``sscan_i8_quant`` gives it) and residual, the sum s (want_residual, by default when a
    residual is given; residual_dtype: its type without one, default x's), and nothing else.
    ``out`` may supply tensors by name; those that are not wanted are neither written nor
    returned; out["residual"] may be residual itself."""
    rows, dim = _tokens(x, "x")
    dt = _float(x, "x")
    shape, dtype = x.shape, x.dtype
    if residual is not None:
        if residual_dtype not in (None, residual.dtype):
            raise ValueError(f"residual must be {residual_dtype}, got {residual.dtype}")
        residual_dtype = residual.dtype
    elif residual_dtype is None:
        residual_dtype = dtype
    if residual_dtype not in (_F32, dtype):
        raise ValueError("the residual must be float32 or of x's type")
    if want_residual is None:
        want_residual = residual is not None
    px, sx = _rows(x, "x", dtype, shape)
    pres, pw = _at(residual, "residual", residual_dtype, shape), _at(weight, "weight", _F32, (dim,))
    get = out.get if out else {}.get
    out = {}                          # a given tensor that is not written has no place in it
    y = py = kept = pk = codes = pc = scales = psc = None
    sc = dim
    if want_y:
        y, py = _new(x, dtype, get("y"), "y")
        out["y"] = y
    if want_residual:
        kept, pk = _new(x, residual_dtype, get("residual"), "residual")
        out["residual"] = kept
    if want_codes:
        codes, pc, sc = _codes(x, get("codes"))
        scales, psc = _scales(x, get("scales"))
        out["codes"], out["scales"] = codes, scales
    _together(x, residual, weight, y, kept, codes, scales)
    _run(x, _lib.sscan_rms_fwd, rows, dim, dt, _DTYPES[residual_dtype], px, sx, pres, pw, eps, py, pk, pc, sc, psc)
    if want_codes and dim == 0:       # rows without channels have scales all the same
        _run(x, _lib.sscan_i8_quant, rows, 0, dt, None, 0, None, 0, psc)
    return out


def sscan_rms_bwd(s: torch.Tensor, weight: Optional[torch.Tensor], dy: torch.Tensor,
                  dresidual: Optional[torch.Tensor] = None, eps: float = 1e-5, want_dx: bool = True,
                  want_dresidual: bool = False, want_dweight: Optional[bool] = None, out: Optional[dict] = None,
                  workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``sscan_rms_fwd``, given dy and, optionally, dresidual, the gradient
    of the sum s from what follows (of s's type).  s: the sum that the forward kept, or x
    itself without a residual.  Returns a dict with dx (dy's type), dresidual (the same
    gradient in s's type, want_dresidual) and dweight (by default when a weight is given), and
    nothing else; ``out`` may supply tensors by name, of which those that are not wanted are
    neither written nor returned; dx also as columns of a wider tensor, out["dresidual"] as
    dresidual itself."""
    rows, dim = _tokens(dy, "dy")
    dt = _float(dy, "dy")
    shape, dtype, kept = dy.shape, dy.dtype, s.dtype
    if kept not in (_F32, dtype):
        raise ValueError("s must be float32 or of dy's type")
    if want_dweight is None:
        want_dweight = weight is not None
    ps, ss = _rows(s, "s", kept, shape)
    pw, pdy, pdk = _at(weight, "weight", _F32, (dim,)), _at(dy, "dy", dtype, shape), _at(dresidual, "dresidual", kept, shape)
    get = out.get if out else {}.get
    out = {}                          # a given tensor that is not written has no place in it
    dx = dres = dw = ws = None
    pdx, sdx = None, dim
    if want_dx:
        dx = get("dx")
        if dx is None:
            dx = torch.empty_like(dy)
        out["dx"] = dx
        pdx, sdx = _rows(dx, "dx", dtype, shape)
    if want_dresidual:
        dres = get("dresidual")
        if dres is None:
            dres = torch.empty(shape, dtype=kept, device=dy.device)
        out["dresidual"] = dres
    pws = nws = None
    if want_dweight:
        dw = get("dweight")
        if dw is None:
            dw = torch.empty(dim, dtype=_F32, device=dy.device)
        out["dweight"] = dw
        ws, pws, nws = _scratch(workspace, _lib.sscan_rms_bwd_workspace_size(rows, dim), dy.device)
    _together(dy, s, weight, dresidual, dx, dres, dw, ws)
    _run(dy, _lib.sscan_rms_bwd, rows, dim, dt, _DTYPES[kept], ps, ss, pw, eps, pdy, pdk, pdx, sdx,
         _at(dres, "dresidual", kept, shape), _at(dw, "dweight", _F32, (dim,)), pws, nws or 0)
    return out


def sscan_i8_quant(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of x [rows, dim] or [batch, seqlen, dim] in 8-bit integers: scale = max|x| / 127 of
    the row (at least 2^-126), code = the whole number nearest to x / scale.  Returns codes
    (int8, x's shape, rows starting at multiples of 16 bytes) and scales (float32, x's shape
    without its last dimension)."""
    rows, dim = _tokens(x, "x")
    dt = _float(x, "x")
    px, sx = _rows(x, "x", x.dtype, x.shape)
    codes, pc, sc = _codes(x, codes)
    scales, ps = _scales(x, scales)
    _together(x, codes, scales)
    _run(x, _lib.sscan_i8_quant, rows, dim, dt, px, sx, pc, sc, ps)
    return codes, scales


def sscan_i8_matmul(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a b^T of rows in 8-bit integers with the scales of both sides: out[..., j] = a_scale
    b_scale[j] (a . b[j]) + bias[j].  a: [rows, k] or [batch, seqlen, k] int8 with a_scales of
    its shape without k; b: [n, k] int8 with b_scales [n]; bias [n] float32.  Returns [..., n]
    of dtype float32 or bfloat16 (``out`` may supply it, also as columns of a wider tensor)."""
    m, k = _tokens(a, "a")
    if b.dim() != 2:
        raise ValueError("b must be [n, k]")
    n = b.shape[0]
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    lead = a.shape[:-1]
    pa, sa = _rows(a, "a", _I8, a.shape)
    pb, sb = _rows(b, "b", _I8, (n, k))
    if out is None:
        out = a.new_empty((m, n) if len(lead) == 1 else (*lead, n), dtype=dtype)
        po, so = out.data_ptr(), n
    else:
        po, so = _rows(out, "out", dtype, (*lead, n))
    _together(a, a_scales, b, b_scales, bias, out)
    _run(a, _lib.sscan_i8_matmul, m, n, k, pa, sa, _at(a_scales, "a_scales", _F32, lead), pb, sb,
         _at(b_scales, "b_scales", _F32, (n,)), _at(bias, "bias", _F32, (n,)), _DTYPES[dtype], po, so)
    return out


def dwconv_bwd_workspace_size(batch: int, seqlen: int, dim: int, dconv: int) -> int:
    return int(_lib.sscan_dwconv_bwd_workspace_size(batch, seqlen, dim, dconv))


def _taps(conv_w: torch.Tensor, dim: int) -> int:
    if conv_w.dim() != 2 or conv_w.shape[0] != dim:
        raise ValueError(f"conv_w must be [{dim}, dconv], got {tuple(conv_w.shape)}")
    return conv_w.shape[1]


def sscan_dwconv_fwd(x: torch.Tensor, conv_w: torch.Tensor, conv_b: Optional[torch.Tensor] = None, silu: bool = True,
                     initial_state: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                     return_last_state: bool = False, out: Optional[torch.Tensor] = None,
                     last_state: Optional[torch.Tensor] = None):
    """Depthwise causal convolution over time, then (silu) SiLU: x [batch, seqlen, dim] (float32
    or bfloat16, dense or columns of a wider tensor), conv_w [dim, dconv], conv_b [dim] float32,
    conv_w[:, -1] on the current token.  offsets [sequences + 1] (int32, on the GPU): batch is 1
    and its tokens are packed requests, the rest padding.  initial_state, last_state: [batch or
    sequences, dim, dconv - 1] float32, the raw inputs before and after.  Returns y, or
    (y, last_state)."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    dt = _float(x, "x")
    batch, seqlen, dim = shape = x.shape
    px, sx = _rows(x, "x", x.dtype, shape)
    taps = _taps(conv_w, dim)
    poff, nseq = _nseq(offsets, batch)
    per_seq = (nseq, dim, max(taps - 1, 0))
    y = _dense_like(x) if out is None else out
    if last_state is None and return_last_state:
        last_state = torch.empty(per_seq, dtype=_F32, device=x.device)
    _together(x, conv_w, conv_b, initial_state, offsets, y, last_state)
    _run(x, _lib.sscan_dwconv_fwd, batch, seqlen, dim, taps, dt, int(silu), px, sx, _at(conv_w, "conv_w", _F32, (dim, taps)),
         _at(conv_b, "conv_b", _F32, (dim,)), _at(initial_state, "initial_state", _F32, per_seq), poff, nseq,
         _at(y, "out", x.dtype, shape), _at(last_state, "last_state", _F32, per_seq))
    return (y, last_state) if return_last_state else y


def sscan_dwconv_bwd(x: torch.Tensor, conv_w: torch.Tensor, dy: torch.Tensor, conv_b: Optional[torch.Tensor] = None,
                     silu: bool = True, initial_state: Optional[torch.Tensor] = None,
                     offsets: Optional[torch.Tensor] = None, dlast_state: Optional[torch.Tensor] = None,
                     want_dbias: bool = True, want_dinitial_state: bool = True, out: Optional[dict] = None,
                     workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``sscan_dwconv_fwd`` for the same inputs, given dy and optionally
    dlast_state.  Returns a dict with dx, dconv_w and, if wanted, dconv_b and dinitial_state;
    ``out`` may supply tensors by name, dx also as columns of a wider tensor."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    dt = _float(x, "x")
    batch, seqlen, dim = shape = x.shape
    dev = x.device
    px, sx = _rows(x, "x", x.dtype, shape)
    taps = _taps(conv_w, dim)
    poff, nseq = _nseq(offsets, batch)
    per_seq = (nseq, dim, max(taps - 1, 0))
    pdy = _at(dy, "dy", x.dtype, shape)
    out = dict(out) if out else {}
    dx, dw, db, dh0 = out.get("dx"), out.get("dconv_w"), out.get("dconv_b"), out.get("dinitial_state")
    if dx is None:
        dx = out["dx"] = _dense_like(x)
    if dw is None:
        dw = out["dconv_w"] = torch.empty((dim, taps), dtype=_F32, device=dev)
    if want_dbias and db is None:
        db = out["dconv_b"] = torch.empty(dim, dtype=_F32, device=dev)
    if want_dinitial_state and dh0 is None:
        dh0 = out["dinitial_state"] = torch.empty(per_seq, dtype=_F32, device=dev)
    pdx, sdx = _rows(dx, "dx", x.dtype, shape)
    ws, pws, nws = _scratch(workspace, _lib.sscan_dwconv_bwd_workspace_size(batch, seqlen, dim, taps), dev)
    _together(x, conv_w, dy, conv_b, initial_state, offsets, dlast_state, dx, dw, db, dh0, ws)
    _run(x, _lib.sscan_dwconv_bwd, batch, seqlen, dim, taps, dt, int(silu), px, sx, _at(conv_w, "conv_w", _F32, (dim, taps)),
         _at(conv_b, "conv_b", _F32, (dim,)), _at(initial_state, "initial_state", _F32, per_seq), poff, nseq, pdy,
         _at(dlast_state, "dlast_state", _F32, per_seq), pdx, sdx, _at(dw, "dconv_w", _F32, (dim, taps)),
         _at(db, "dconv_b", _F32, (dim,)), _at(dh0, "dinitial_state", _F32, per_seq), pws, nws)
    return out


def sscan_dwconv_step(state: torch.Tensor, x: torch.Tensor, conv_w: torch.Tensor, conv_b: Optional[torch.Tensor] = None,
                      silu: bool = True, slots: Optional[torch.Tensor] = None, slots_out: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the convolution for every row of a batch.  state: [slots, dim, dconv - 1]
    float32, a pool updated in place; x: [batch, dim]; slots [batch] (int32): row b continues
    state slots[b] (none and y = 0 if negative), default slot b; slots_out [batch] (int32):
    where its new state goes, default its own slot.  Returns y [batch, dim]."""
    if x.dim() != 2:
        raise ValueError("x must be [batch, dim]")
    dt = _float(x, "x")
    batch, dim = shape = x.shape
    px, sx = _rows(x, "x", x.dtype, shape)
    taps = _taps(conv_w, dim)
    if state.dim() != 3:
        raise ValueError("state must be [slots, dim, dconv - 1]")
    pool = state.shape[0]
    y = _dense_like(x) if out is None else out
    _together(x, state, conv_w, conv_b, slots, slots_out, y)
    _run(x, _lib.sscan_dwconv_step, batch, dim, taps, dt, int(silu), _at(state, "state", _F32, (pool, dim, max(taps - 1, 0))),
         pool, _at(slots, "slots", torch.int32, (batch,)), _at(slots_out, "slots_out", torch.int32, (batch,)), px, sx,
         _at(conv_w, "conv_w", _F32, (dim, taps)), _at(conv_b, "conv_b", _F32, (dim,)), _at(y, "out", x.dtype, shape))
    return y
