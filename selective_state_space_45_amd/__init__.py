"""Python binding of libselscan: the selective state-space scan on MI355X (gfx950).

Argument marshalling only: every step of the scan runs in the HIP kernels of
``libselscan.so`` (see ``include/selscan.h`` for the operation and its sources on
the reference pages).  PyTorch supplies device memory and the current stream.
There is no fallback: if the library is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libselscan.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libselscan.so not found at {LIB_PATH}; build it with "
        "`python -m selective_state_space_45_amd.build` (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t

_lib.sscan_version.argtypes = []
_lib.sscan_version.restype = ctypes.c_int
_lib.sscan_last_error.argtypes = []
_lib.sscan_last_error.restype = ctypes.c_char_p
_lib.sscan_fwd_workspace_size.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int]
_lib.sscan_fwd_workspace_size.restype = _SZ
_lib.sscan_fwd_segmented_workspace_size.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _I64]
_lib.sscan_fwd_segmented_workspace_size.restype = _SZ
_U32 = ctypes.c_uint
_lib.sscan_fwd.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 11 + [_P, _SZ, _P]
_lib.sscan_fwd.restype = ctypes.c_int
_lib.sscan_fwd_segmented.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 11 + [_P, _SZ, _I64, _P]
_lib.sscan_fwd_segmented.restype = ctypes.c_int
_lib.sscan_fwd_noalloc.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 11 + [_P]
_lib.sscan_fwd_noalloc.restype = ctypes.c_int
_lib.sscan_step.argtypes = [_I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 11
_lib.sscan_step.restype = ctypes.c_int
_lib.sscan_fwd_conv.argtypes = [_I64, _I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 15 + [_P, _SZ, _P]
_lib.sscan_fwd_conv.restype = ctypes.c_int
_lib.sscan_step_conv.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 14
_lib.sscan_step_conv.restype = ctypes.c_int
_lib.sscan_bwd_workspace_size.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int]
_lib.sscan_bwd_workspace_size.restype = _SZ
_lib.sscan_bwd.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 21 + [_SZ, _P]
_lib.sscan_bwd.restype = ctypes.c_int
_lib.sscan_checkpoint_bytes.argtypes = [_I64, _I64, _I64, _I64]
_lib.sscan_checkpoint_bytes.restype = _SZ
_lib.sscan_fwd_checkpointed.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 11 + [_P, _SZ, _P, _SZ, _P]
_lib.sscan_fwd_checkpointed.restype = ctypes.c_int
_lib.sscan_bwd_checkpointed_workspace_size.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int]
_lib.sscan_bwd_checkpointed_workspace_size.restype = _SZ
_lib.sscan_bwd_checkpointed.argtypes = ([_I64, _I64, _I64, _I64, ctypes.c_int, _U32] + [_P] * 8 + [_P, _SZ] + [_P] * 11
                                        + [_P, _SZ, _P])
_lib.sscan_bwd_checkpointed.restype = ctypes.c_int

SSCAN_F32, SSCAN_BF16 = 0, 1
SSCAN_FLAG_EULER = 1
SSCAN_FLAG_STRUCTURED_A = 2
_DTYPES = {torch.float32: SSCAN_F32, torch.bfloat16: SSCAN_BF16}
STATUS = {0: "SSCAN_OK", 1: "SSCAN_ERR_INVALID_ARG", 2: "SSCAN_ERR_UNSUPPORTED", 3: "SSCAN_ERR_HIP"}


class SelScanError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


def version() -> int:
    return int(_lib.sscan_version())


def last_error() -> str:
    return _lib.sscan_last_error().decode()


def library():
    """The loaded ctypes library (for callers that marshal pointers themselves)."""
    return _lib


def _check(rc: int):
    if rc != 0:
        raise SelScanError(rc, last_error())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _stream(dev) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def fwd_workspace_size(batch: int, seqlen: int, dim: int, dstate: int, dtype=torch.bfloat16,
                       num_segments: Optional[int] = None) -> int:
    """Workspace bytes for the automatic split, or for num_segments segments."""
    if num_segments is not None:
        return int(_lib.sscan_fwd_segmented_workspace_size(batch, seqlen, dim, dstate, _DTYPES[dtype], num_segments))
    return int(_lib.sscan_fwd_workspace_size(batch, seqlen, dim, dstate, _DTYPES[dtype]))


def sscan_fwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
              D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
              delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
              return_last_state: bool = False, out: Optional[torch.Tensor] = None,
              last_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              num_segments: Optional[int] = None, euler: bool = False,
              conv_w: Optional[torch.Tensor] = None, conv_b: Optional[torch.Tensor] = None,
              conv_state_in: Optional[torch.Tensor] = None, conv_state_out: Optional[torch.Tensor] = None,
              checkpoints: Optional[torch.Tensor] = None, structured_a: bool = False):
    """Forward selective scan.  x, delta, z: [batch, seqlen, dim]; B, C: [batch, seqlen, dstate]
    (all float32 or all bfloat16); A: [dim, dstate], D, delta_bias: [dim], initial_state:
    [batch, dim, dstate] (float32).  euler: Bbar = Delta B instead of the zero-order hold.
    conv_w [dim, dconv] (float32): x is the raw input of the fused causal depthwise
    convolution + SiLU prologue (conv_b [dim], conv_state_in / conv_state_out
    [batch, dim, dconv - 1], float32, optional).  checkpoints (a device buffer of at least
    ``checkpoint_bytes(...)`` bytes): also save the states that ``sscan_bwd(...,
    checkpoints=...)`` starts from.  structured_a: the caller states A[d, n] = c_d a_n
    (SSCAN_FLAG_STRUCTURED_A, a hint the library verifies).  Returns y, or (y, last_state)."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    batch, seqlen, dim = x.shape
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    dt = _DTYPES[x.dtype]
    dstate = A.shape[1] if A.dim() == 2 else -1
    _dev(x, "x")
    _dev(delta, "delta", x.dtype, x.shape)
    _dev(A, "A", torch.float32, (dim, dstate))
    _dev(B, "B", x.dtype, (batch, seqlen, dstate))
    _dev(C, "C", x.dtype, (batch, seqlen, dstate))
    if D is not None:
        _dev(D, "D", torch.float32, (dim,))
    if z is not None:
        _dev(z, "z", x.dtype, x.shape)
    if delta_bias is not None:
        _dev(delta_bias, "delta_bias", torch.float32, (dim,))
    if initial_state is not None:
        _dev(initial_state, "initial_state", torch.float32, (batch, dim, dstate))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", x.dtype, x.shape)
    ls = last_state
    if ls is None and return_last_state:
        ls = torch.empty((batch, dim, dstate), dtype=torch.float32, device=x.device)
    if ls is not None:
        _dev(ls, "last_state", torch.float32, (batch, dim, dstate))
    if workspace is None:
        need = fwd_workspace_size(batch, seqlen, dim, dstate, x.dtype, num_segments)
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device) if need > 0 else None
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    flags = (SSCAN_FLAG_EULER if euler else 0) | (SSCAN_FLAG_STRUCTURED_A if structured_a else 0)
    args = [batch, seqlen, dim, dstate, dt, flags, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
            _ptr(delta_bias), _ptr(initial_state), _ptr(y), _ptr(ls), _ptr(workspace), wbytes]
    if conv_w is not None:
        if num_segments is not None:
            raise ValueError("num_segments is not available with the convolution prologue")
        if checkpoints is not None:
            raise ValueError("checkpoints are not available with the convolution prologue")
        dconv = conv_w.shape[1] if conv_w.dim() == 2 else -1
        _dev(conv_w, "conv_w", torch.float32, (dim, dconv))
        if conv_b is not None:
            _dev(conv_b, "conv_b", torch.float32, (dim,))
        for t, name in ((conv_state_in, "conv_state_in"), (conv_state_out, "conv_state_out")):
            if t is not None:
                _dev(t, name, torch.float32, (batch, dim, dconv - 1))
        cargs = [batch, seqlen, dim, dstate, dconv, dt, flags, _ptr(x), _ptr(conv_w), _ptr(conv_b),
                 _ptr(conv_state_in), _ptr(conv_state_out)] + args[7:]
        _check(_lib.sscan_fwd_conv(*cargs, _stream(x.device)))
    elif checkpoints is not None:
        if num_segments is not None:
            raise ValueError("num_segments is not available with checkpoints")
        _dev(checkpoints, "checkpoints")
        _check(_lib.sscan_fwd_checkpointed(*args, _ptr(checkpoints),
                                           checkpoints.numel() * checkpoints.element_size(), _stream(x.device)))
    elif num_segments is None:
        _check(_lib.sscan_fwd(*args, _stream(x.device)))
    else:
        _check(_lib.sscan_fwd_segmented(*args, int(num_segments), _stream(x.device)))
    if return_last_state:
        return y, ls
    return y


def sscan_fwd_noalloc(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                      D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                      delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, last_state: Optional[torch.Tensor] = None,
                      euler: bool = False) -> torch.Tensor:
    """``sscan_fwd`` for callers that cannot allocate: the library's static device
    scratch replaces the workspace.  ``out`` (and ``last_state`` if wanted) must be
    given, so this call allocates nothing either.  Returns ``out``."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    if out is None:
        raise ValueError("out is required (the no-allocation path allocates nothing)")
    batch, seqlen, dim = x.shape
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    dstate = A.shape[1] if A.dim() == 2 else -1
    _dev(x, "x")
    _dev(delta, "delta", x.dtype, x.shape)
    _dev(A, "A", torch.float32, (dim, dstate))
    _dev(B, "B", x.dtype, (batch, seqlen, dstate))
    _dev(C, "C", x.dtype, (batch, seqlen, dstate))
    for t, name, shape in ((D, "D", (dim,)), (delta_bias, "delta_bias", (dim,)),
                           (initial_state, "initial_state", (batch, dim, dstate)),
                           (last_state, "last_state", (batch, dim, dstate))):
        if t is not None:
            _dev(t, name, torch.float32, shape)
    if z is not None:
        _dev(z, "z", x.dtype, x.shape)
    _dev(out, "out", x.dtype, x.shape)
    flags = SSCAN_FLAG_EULER if euler else 0
    _check(_lib.sscan_fwd_noalloc(batch, seqlen, dim, dstate, _DTYPES[x.dtype], flags, _ptr(x), _ptr(delta),
                                  _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
                                  _ptr(initial_state), _ptr(out), _ptr(last_state), _stream(x.device)))
    return out


def sscan_step(state: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
               C: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
               delta_bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               euler: bool = False, conv_w: Optional[torch.Tensor] = None, conv_b: Optional[torch.Tensor] = None,
               conv_state: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step.  state: [batch, dim, dstate] float32, updated in place; x, delta, z:
    [batch, dim]; B, C: [batch, dstate] (float32 or bfloat16); A: [dim, dstate].  euler: Bbar =
    Delta B instead of the zero-order hold.  conv_w [dim, dconv]: x is a raw input of the
    convolution prologue whose cache conv_state [batch, dim, dconv - 1] (float32) is
    updated in place.  Returns y [batch, dim]."""
    if x.dim() != 2:
        raise ValueError("x must be [batch, dim]")
    batch, dim = x.shape
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    dstate = A.shape[1] if A.dim() == 2 else -1
    _dev(state, "state", torch.float32, (batch, dim, dstate))
    _dev(x, "x")
    _dev(delta, "delta", x.dtype, x.shape)
    _dev(A, "A", torch.float32, (dim, dstate))
    _dev(B, "B", x.dtype, (batch, dstate))
    _dev(C, "C", x.dtype, (batch, dstate))
    if D is not None:
        _dev(D, "D", torch.float32, (dim,))
    if z is not None:
        _dev(z, "z", x.dtype, x.shape)
    if delta_bias is not None:
        _dev(delta_bias, "delta_bias", torch.float32, (dim,))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", x.dtype, x.shape)
    flags = SSCAN_FLAG_EULER if euler else 0
    if conv_w is not None:
        dconv = conv_w.shape[1] if conv_w.dim() == 2 else -1
        _dev(conv_w, "conv_w", torch.float32, (dim, dconv))
        if conv_b is not None:
            _dev(conv_b, "conv_b", torch.float32, (dim,))
        if conv_state is not None:
            _dev(conv_state, "conv_state", torch.float32, (batch, dim, dconv - 1))
        _check(_lib.sscan_step_conv(batch, dim, dstate, dconv, _DTYPES[x.dtype], flags, _ptr(state),
                                    _ptr(conv_state), _ptr(x), _ptr(conv_w), _ptr(conv_b), _ptr(delta), _ptr(A),
                                    _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias), _ptr(y),
                                    _stream(x.device)))
        return y
    _check(_lib.sscan_step(batch, dim, dstate, _DTYPES[x.dtype], flags, _ptr(state), _ptr(x), _ptr(delta),
                           _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias), _ptr(y),
                           _stream(x.device)))
    return y


def bwd_workspace_size(batch: int, seqlen: int, dim: int, dstate: int, dtype=torch.bfloat16,
                       checkpointed: bool = False) -> int:
    fn = _lib.sscan_bwd_checkpointed_workspace_size if checkpointed else _lib.sscan_bwd_workspace_size
    return int(fn(batch, seqlen, dim, dstate, _DTYPES[dtype]))


def checkpoint_bytes(batch: int, seqlen: int, dim: int, dstate: int) -> int:
    """Bytes of the checkpoint buffer for ``sscan_fwd(..., checkpoints=...)`` and
    ``sscan_bwd(..., checkpoints=...)``: the state entering every 8 timesteps,
    [batch, ceil(seqlen / 8), dstate, dim] float32."""
    return int(_lib.sscan_checkpoint_bytes(batch, seqlen, dim, dstate))


def sscan_bwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
              dy: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
              delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
              dlast_state: Optional[torch.Tensor] = None, euler: bool = False,
              want_ddelta_bias: bool = True, want_dinitial_state: bool = True,
              workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None,
              checkpoints: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``sscan_fwd``: gradients of a scalar loss given dy = dLoss/dy
    (same shape and dtype as x) and optionally dlast_state = dLoss/d(last state).
    Returns a dict with dx, ddelta, dA, dB, dC and, as applicable, dD, dz,
    ddelta_bias, dinitial_state (``out`` may supply preallocated tensors by name).
    checkpoints: the buffer ``sscan_fwd(..., checkpoints=...)`` filled for the same
    inputs; the forward recurrence is then not run again (initial_state then enters
    through the checkpoints and is not needed)."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    batch, seqlen, dim = x.shape
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    dstate = A.shape[1] if A.dim() == 2 else -1
    _dev(x, "x")
    _dev(delta, "delta", x.dtype, x.shape)
    _dev(dy, "dy", x.dtype, x.shape)
    _dev(A, "A", torch.float32, (dim, dstate))
    _dev(B, "B", x.dtype, (batch, seqlen, dstate))
    _dev(C, "C", x.dtype, (batch, seqlen, dstate))
    for t, name, shape in ((D, "D", (dim,)), (delta_bias, "delta_bias", (dim,)),
                           (initial_state, "initial_state", (batch, dim, dstate)),
                           (dlast_state, "dlast_state", (batch, dim, dstate))):
        if t is not None:
            _dev(t, name, torch.float32, shape)
    if z is not None:
        _dev(z, "z", x.dtype, x.shape)
    out = dict(out or {})
    dev = x.device

    def get(name, shape, dtype):
        t = out.get(name)
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
            out[name] = t
        return _dev(t, name, dtype, shape)

    dx = get("dx", x.shape, x.dtype)
    ddelta = get("ddelta", x.shape, x.dtype)
    dA = get("dA", (dim, dstate), torch.float32)
    dB = get("dB", (batch, seqlen, dstate), x.dtype)
    dC = get("dC", (batch, seqlen, dstate), x.dtype)
    dD = get("dD", (dim,), torch.float32) if D is not None else None
    dz = get("dz", x.shape, x.dtype) if z is not None else None
    dbias = get("ddelta_bias", (dim,), torch.float32) if want_ddelta_bias else None
    dh0 = get("dinitial_state", (batch, dim, dstate), torch.float32) if want_dinitial_state else None
    need = bwd_workspace_size(batch, seqlen, dim, dstate, x.dtype, checkpointed=checkpoints is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    wbytes = workspace.numel() * workspace.element_size()
    flags = SSCAN_FLAG_EULER if euler else 0
    if checkpoints is not None:
        _dev(checkpoints, "checkpoints")
        _check(_lib.sscan_bwd_checkpointed(
            batch, seqlen, dim, dstate, _DTYPES[x.dtype], flags, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
            _ptr(D), _ptr(z), _ptr(delta_bias), _ptr(checkpoints), checkpoints.numel() * checkpoints.element_size(),
            _ptr(dy), _ptr(dlast_state), _ptr(dx), _ptr(ddelta), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dz),
            _ptr(dbias), _ptr(dh0), _ptr(workspace), wbytes, _stream(dev)))
        return out
    _check(_lib.sscan_bwd(batch, seqlen, dim, dstate, _DTYPES[x.dtype], flags, _ptr(x), _ptr(delta), _ptr(A),
                          _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias), _ptr(initial_state), _ptr(dy),
                          _ptr(dlast_state), _ptr(dx), _ptr(ddelta), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD),
                          _ptr(dz), _ptr(dbias), _ptr(dh0), _ptr(workspace), wbytes, _stream(dev)))
    return out


# ---------------------------------------------------------------------------
# Gated linear recurrence, and activations in 8 bits
# ---------------------------------------------------------------------------
_F = ctypes.c_float
_I = ctypes.c_int
for _name, _args, _res in (
        ("sscan_act8_bytes", [_I64] * 3, _SZ),
        ("sscan_act8_pack", [_I64] * 3 + [_I, _P, _I64, _P, _SZ, _P], _I),
        ("sscan_act8_unpack", [_I64] * 3 + [_I, _P, _SZ, _P, _P], _I),
        ("sscan_glr_checkpoint_bytes", [_I64] * 3, _SZ),
        ("sscan_glr_saved_bytes", [_I64] * 3 + [_I], _SZ),
        ("sscan_glr_fwd_workspace_size", [_I64] * 3, _SZ),
        ("sscan_glr_bwd_workspace_size", [_I64] * 3, _SZ),
        ("sscan_glr_fwd", [_I64] * 3 + [_I] + [_P] * 8 + [_F, _P, _P, _I64] + [_P] * 3 + [_SZ, _P, _SZ, _P, _SZ, _P], _I),
        ("sscan_glr_bwd", [_I64] * 3 + [_I] + [_P] * 6 + [_SZ] + [_P] * 3 + [_F, _P, _P, _I64, _P, _SZ] + [_P] * 12
         + [_SZ, _P], _I),
        ("sscan_glr_step", [_I64] * 2 + [_I, _P, _I64] + [_P] * 10 + [_F, _P, _P], _I)):
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _res


# The calls below are made once a token in a decode loop, where the host's time counts:
# a good argument costs one helper call, and the messages are made only for a bad one.

def _rows(t: torch.Tensor, name: str, dtype, shape):
    """(address, token stride in elements) of a token tensor, whose rows may be columns of a
    wider one (last index dense, tokens evenly spaced)."""
    if t.is_cuda and t.dtype is dtype and t.shape == shape:
        if t.is_contiguous():
            return t.data_ptr(), shape[-1]
        st = t.stride()
        step, even = st[-2], len(shape) == 2 or shape[0] == 1 or st[0] == shape[1] * st[-2]
        if len(shape) == 3 and shape[1] == 1:
            step, even = st[0], True
        if (st[-1] == 1 or shape[-1] == 1) and even and step >= shape[-1]:
            return t.data_ptr(), step
        raise ValueError(f"{name} must have a dense last dimension and evenly spaced tokens, got strides {st}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _at(t: Optional[torch.Tensor], name: str, dtype, shape):
    """The address of a dense tensor (None for None)."""
    if t is None:
        return None
    if not (t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _dev(t, name, dtype, shape)
    return t.data_ptr()


def _bytes_at(t: Optional[torch.Tensor], name: str):
    """(address, bytes) of a dense buffer of any type ((None, 0) for None)."""
    if t is None:
        return None, 0
    if not (t.is_cuda and t.is_contiguous()):
        _dev(t, name)
    return t.data_ptr(), t.numel() * t.element_size()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_at(t: torch.Tensor):
    """The handle of the current stream of t's device."""
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _dense_like(x: torch.Tensor) -> torch.Tensor:
    """A dense tensor of x's shape (empty_like is the cheaper call, where it gives that)."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _strides(values, dim: int):
    for v in values:
        if v != dim:
            return (ctypes.c_int64 * 4)(*values)
    return None


def _nseq(offsets, batch):
    """(address of offsets, number of sequences)."""
    if offsets is None:
        return None, batch
    _dev(offsets, "offsets", torch.int32)
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be [sequences + 1]")
    return offsets.data_ptr(), offsets.numel() - 1


def _scratch(workspace, need, device):
    """A workspace of `need` bytes unless one was given, with its address and size."""
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return (workspace,) + _bytes_at(workspace, "workspace")


def act8_bytes(batch: int, seqlen: int, dim: int) -> int:
    """Bytes of one activation tensor [batch, seqlen, dim] packed to 8 bits."""
    return int(_lib.sscan_act8_bytes(batch, seqlen, dim))


def sscan_act8_pack(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [batch, seqlen, dim] (float32 or bfloat16, tokens evenly spaced) in 8 bits: every
    channel's 16 consecutive tokens share a power of two.  Returns a byte tensor of
    ``act8_bytes`` bytes (``out`` may supply it)."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    batch, seqlen, dim = x.shape
    at, stride = _rows(x, "x", x.dtype, x.shape)
    if out is None:
        out = torch.empty(act8_bytes(batch, seqlen, dim), dtype=torch.uint8, device=x.device)
    to, size = _bytes_at(out, "out")
    _check(_lib.sscan_act8_pack(batch, seqlen, dim, _DTYPES[x.dtype], at, stride, to, size, _stream_at(x)))
    return out


def sscan_act8_unpack(packed: torch.Tensor, shape, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None
                      ) -> torch.Tensor:
    """The values of a tensor that ``sscan_act8_pack`` packed, as ``dtype`` of the given
    shape [batch, seqlen, dim] (``out`` may supply the tensor)."""
    if len(shape) != 3:
        raise ValueError("shape must be [batch, seqlen, dim]")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    at, size = _bytes_at(packed, "packed")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=packed.device)
    _check(_lib.sscan_act8_unpack(shape[0], shape[1], shape[2], _DTYPES[dtype], at, size,
                                  _at(out, "out", dtype, torch.Size(shape)), _stream_at(packed)))
    return out


def glr_checkpoint_bytes(batch: int, seqlen: int, dim: int) -> int:
    """Bytes of the states ``sscan_glr_fwd`` keeps for the backward pass (one every 64
    tokens, [batch, ceil(seqlen / 64), dim] float32)."""
    return int(_lib.sscan_glr_checkpoint_bytes(batch, seqlen, dim))


def glr_saved_bytes(batch: int, seqlen: int, dim: int, gated: bool = False) -> int:
    """Bytes of the activations (x, r, i and, if gated, z) saved in 8 bits."""
    return int(_lib.sscan_glr_saved_bytes(batch, seqlen, dim, int(gated)))


def glr_workspace_size(batch: int, seqlen: int, dim: int, backward: bool = False) -> int:
    fn = _lib.sscan_glr_bwd_workspace_size if backward else _lib.sscan_glr_fwd_workspace_size
    return int(fn(batch, seqlen, dim))


def sscan_glr_fwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, lam: torch.Tensor,
                  r_bias: Optional[torch.Tensor] = None, i_bias: Optional[torch.Tensor] = None,
                  z: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                  offsets: Optional[torch.Tensor] = None, decay_scale: float = 8.0, return_last_state: bool = False,
                  out: Optional[torch.Tensor] = None, last_state: Optional[torch.Tensor] = None,
                  checkpoints: Optional[torch.Tensor] = None, saved: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None):
    """Gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) (sigmoid(i_t + i_bias) x_t),
    a_t = exp(-decay_scale softplus(lam) sigmoid(r_t + r_bias)); y = h, or h silu(z).

    x, r, i, z: [batch, seqlen, dim] (all float32 or all bfloat16), each dense or columns of a
    wider tensor; lam, r_bias, i_bias: [dim] float32.  offsets [sequences + 1] (int32, on the
    GPU): batch is 1 and its tokens are packed requests, the rest padding.  initial_state,
    last_state: [batch or sequences, dim] float32.  checkpoints (``glr_checkpoint_bytes``
    bytes) and saved (``glr_saved_bytes`` bytes) are filled for ``sscan_glr_bwd``, the latter
    with the activations in 8 bits, whose groups of 16 tokens are cut by position: packed
    requests that meet inside one share its scale, and a NaN.  Returns y, or (y, last_state)."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    batch, seqlen, dim = shape = x.shape
    dtype = x.dtype
    px, sx = _rows(x, "x", dtype, shape)
    pr, sr = _rows(r, "r", dtype, shape)
    pi, si = _rows(i, "i", dtype, shape)
    pz, sz = (None, dim) if z is None else _rows(z, "z", dtype, shape)
    poff, nseq = _nseq(offsets, batch)
    y = _dense_like(x) if out is None else out
    if last_state is None and return_last_state:
        last_state = torch.empty((nseq, dim), dtype=torch.float32, device=x.device)
    workspace, pw, nw = _scratch(workspace, _lib.sscan_glr_fwd_workspace_size(batch, seqlen, dim), x.device)
    f32, per_channel, per_seq = torch.float32, (dim,), (nseq, dim)
    rc = _lib.sscan_glr_fwd(
        batch, seqlen, dim, _DTYPES[dtype], px, pr, pi, pz, _strides((sx, sr, si, sz), dim),
        _at(lam, "lam", f32, per_channel), _at(r_bias, "r_bias", f32, per_channel),
        _at(i_bias, "i_bias", f32, per_channel), decay_scale, _at(initial_state, "initial_state", f32, per_seq), poff, nseq,
        _at(y, "out", dtype, shape), _at(last_state, "last_state", f32, per_seq), *_bytes_at(checkpoints, "checkpoints"),
        *_bytes_at(saved, "saved"), pw, nw, _stream_at(x))
    if rc:
        _check(rc)
    return (y, last_state) if return_last_state else y


def sscan_glr_bwd(lam: torch.Tensor, dy: torch.Tensor, checkpoints: torch.Tensor,
                  x: Optional[torch.Tensor] = None, r: Optional[torch.Tensor] = None,
                  i: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                  saved: Optional[torch.Tensor] = None, gated: bool = False,
                  r_bias: Optional[torch.Tensor] = None, i_bias: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                  decay_scale: float = 8.0, dlast_state: Optional[torch.Tensor] = None, want_dbias: bool = True,
                  want_dinitial_state: bool = True, out: Optional[dict] = None,
                  workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``sscan_glr_fwd``, given dy and what the forward left in
    ``checkpoints``, with either its inputs x, r, i (and z) or the activations it ``saved`` in
    8 bits (``gated`` says whether z is among them).  initial_state is read with offsets only.
    Returns a dict with dx, dr, di, dlam and, as applicable, dz, dr_bias, di_bias,
    dinitial_state; ``out`` may supply tensors by name, the token gradients also as columns of
    a wider tensor."""
    if dy.dim() != 3:
        raise ValueError("dy must be [batch, seqlen, dim]")
    if dy.dtype not in _DTYPES:
        raise ValueError("dy must be float32 or bfloat16")
    batch, seqlen, dim = shape = dy.shape
    dtype, dev = dy.dtype, dy.device
    pdy = _at(dy, "dy", dtype, shape)
    px = pr = pi = pz = None
    sx = sr = si = sz = dim
    if saved is not None:
        if x is not None or r is not None or i is not None or z is not None:
            raise ValueError("give either saved or x, r, i and z")
    else:
        if x is None or r is None or i is None:
            raise ValueError("x, r and i are required without saved")
        if gated and z is None:
            raise ValueError("z is required without saved when gated")
        gated = z is not None
        px, sx = _rows(x, "x", dtype, shape)
        pr, sr = _rows(r, "r", dtype, shape)
        pi, si = _rows(i, "i", dtype, shape)
        if gated:
            pz, sz = _rows(z, "z", dtype, shape)
    poff, nseq = _nseq(offsets, batch)
    out = dict(out or {})
    grads = []
    for name in ("dx", "dr", "di", "dz") if gated else ("dx", "dr", "di"):
        g = out.get(name)
        if g is None:
            g = out[name] = torch.empty_like(dy)
        grads.append(_rows(g, name, dtype, shape))
    if not gated:
        grads.append((None, dim))
    f32, per_channel, per_seq = torch.float32, (dim,), (nseq, dim)
    for name, want, size in (("dlam", True, per_channel), ("dr_bias", want_dbias, per_channel),
                             ("di_bias", want_dbias, per_channel), ("dinitial_state", want_dinitial_state, per_seq)):
        if want and name not in out:
            out[name] = torch.empty(size, dtype=f32, device=dev)
    workspace, pw, nw = _scratch(workspace, _lib.sscan_glr_bwd_workspace_size(batch, seqlen, dim), dev)
    rc = _lib.sscan_glr_bwd(
        batch, seqlen, dim, _DTYPES[dtype], px, pr, pi, pz, _strides((sx, sr, si, sz), dim), *_bytes_at(saved, "saved"),
        _at(lam, "lam", f32, per_channel), _at(r_bias, "r_bias", f32, per_channel),
        _at(i_bias, "i_bias", f32, per_channel), decay_scale, _at(initial_state, "initial_state", f32, per_seq), poff, nseq,
        *_bytes_at(checkpoints, "checkpoints"), pdy,
        _at(dlast_state, "dlast_state", f32, per_seq), grads[0][0], grads[1][0], grads[2][0], grads[3][0],
        _strides([g[1] for g in grads], dim), _at(out["dlam"], "dlam", f32, per_channel),
        _at(out.get("dr_bias"), "dr_bias", f32, per_channel), _at(out.get("di_bias"), "di_bias", f32, per_channel),
        _at(out.get("dinitial_state"), "dinitial_state", f32, per_seq), pw, nw, _stream_at(dy))
    if rc:
        _check(rc)
    return out


def sscan_glr_step(state: torch.Tensor, x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, lam: torch.Tensor,
                   r_bias: Optional[torch.Tensor] = None, i_bias: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                   slots_out: Optional[torch.Tensor] = None, decay_scale: float = 8.0,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the gated linear recurrence for every row of a batch.  state: [slots, dim]
    float32, a pool updated in place; x, r, i, z: [batch, dim]; slots [batch] (int32): row b
    continues state slots[b] (none and y = 0 if negative), default slot b; slots_out [batch]
    (int32): where its new state goes, default its own slot.  Returns y [batch, dim]."""
    if x.dim() != 2:
        raise ValueError("x must be [batch, dim]")
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    batch, dim = shape = x.shape
    dtype = x.dtype
    px, sx = _rows(x, "x", dtype, shape)
    pr, sr = _rows(r, "r", dtype, shape)
    pi, si = _rows(i, "i", dtype, shape)
    pz, sz = (None, dim) if z is None else _rows(z, "z", dtype, shape)
    if state.dim() != 2:
        raise ValueError("state must be [slots, dim]")
    pool = state.shape[0]
    y = _dense_like(x) if out is None else out
    f32, per_channel, per_row = torch.float32, (dim,), (batch,)
    rc = _lib.sscan_glr_step(
        batch, dim, _DTYPES[dtype], _at(state, "state", f32, (pool, dim)), pool, _at(slots, "slots", torch.int32, per_row),
        _at(slots_out, "slots_out", torch.int32, per_row), px, pr, pi, pz, _strides((sx, sr, si, sz), dim),
        _at(lam, "lam", f32, per_channel), _at(r_bias, "r_bias", f32, per_channel),
        _at(i_bias, "i_bias", f32, per_channel), decay_scale, _at(y, "out", dtype, shape), _stream_at(x))
    if rc:
        _check(rc)
    return y


from .layer_ops import *  # noqa: E402,F401,F403  (norm, 8-bit products, convolution: uses what is above)
