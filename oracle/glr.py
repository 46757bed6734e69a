"""Plain float64 forms of the gated linear recurrence and of 8-bit activations, token
after token, for the tests.  Arrays are numpy; nothing here is shared with the kernels.

Dense inputs are [batch, seqlen, dim]; with ``offsets`` the batch is 1 and sequence s is
tokens offsets[s] .. offsets[s + 1], the tokens from offsets[-1] on being padding.
"""
from __future__ import annotations

import numpy as np

BLOCK = 64
GROUP = 16


def _sigmoid(v):
    w = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + w), w / (1.0 + w))


def _sequences(shape, offsets):
    """(row, begin, end) of every sequence."""
    if offsets is None:
        return [(b, 0, shape[1]) for b in range(shape[0])]
    return [(0, int(lo), int(hi)) for lo, hi in zip(offsets[:-1], offsets[1:])]


def _gates(x, r, i, lam, r_bias, i_bias, scale):
    rate = scale * (np.maximum(lam, 0.0) + np.log1p(np.exp(-np.abs(lam))))
    rho = _sigmoid(r if r_bias is None else r + r_bias)
    iota = _sigmoid(i if i_bias is None else i + i_bias)
    return rate, rho, iota, np.exp(-rate * rho), np.sqrt(-np.expm1(-2.0 * rate * rho))


def _f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def fwd(x, r, i, lam, r_bias=None, i_bias=None, z=None, initial_state=None, offsets=None, scale=8.0,
        block_states=None):
    """y, last states [sequences, dim], and the state before each token [batch, seqlen, dim]
    (zero at padding).  block_states: states before the tokens of another run, from which
    every block of 64 tokens starts anew (what a backward pass from 8 bits does)."""
    x, r, i, lam, r_bias, i_bias, z, h0 = _f64(x, r, i, lam, r_bias, i_bias, z, initial_state)
    _, _, iota, a, m = _gates(x, r, i, lam, r_bias, i_bias, scale)
    y, before = np.zeros_like(x), np.zeros_like(x)
    seqs = _sequences(x.shape, offsets)
    last = np.zeros((len(seqs), x.shape[2]))
    gate = None if z is None else z * _sigmoid(z)
    for s, (b, lo, hi) in enumerate(seqs):
        h = np.zeros(x.shape[2]) if h0 is None else h0[s]
        for t in range(lo, hi):
            if block_states is not None and t > lo and t % BLOCK == 0:
                h = block_states[b, t]
            before[b, t] = h
            h = a[b, t] * h + m[b, t] * iota[b, t] * x[b, t]
            y[b, t] = h if gate is None else h * gate[b, t]
        last[s] = h
    return y, last, before


def bwd(x, r, i, lam, dy, r_bias=None, i_bias=None, z=None, initial_state=None, offsets=None, scale=8.0,
        dlast_state=None, before=None):
    """Gradients as a dict.  before: the state before each token (default: the forward's)."""
    if before is None:
        before = fwd(x, r, i, lam, r_bias, i_bias, z, initial_state, offsets, scale)[2]
    x, r, i, lam, r_bias, i_bias, z, dy, dlast = _f64(x, r, i, lam, r_bias, i_bias, z, dy, dlast_state)
    rate, rho, iota, a, m = _gates(x, r, i, lam, r_bias, i_bias, scale)
    out = {k: np.zeros_like(x) for k in ("dx", "dr", "di")}
    if z is not None:
        out["dz"] = np.zeros_like(x)
    seqs = _sequences(x.shape, offsets)
    out["dinitial_state"] = np.zeros((len(seqs), x.shape[2]))
    dlam = np.zeros(x.shape[2])
    for s, (b, lo, hi) in enumerate(seqs):
        g = np.zeros(x.shape[2]) if dlast is None else dlast[s]
        for t in range(hi - 1, lo - 1, -1):
            A, M, P, I, X, H = a[b, t], m[b, t], rho[b, t], iota[b, t], x[b, t], before[b, t]
            gy = dy[b, t]
            if z is not None:
                sz = _sigmoid(z[b, t])
                out["dz"][b, t] = gy * (A * H + M * I * X) * (sz + z[b, t] * sz * (1.0 - sz))
                gy = gy * z[b, t] * sz
            g = g + gy
            dlog = g * (A * H - I * X * A * A / np.where(M > 0, M, np.inf))
            out["dx"][b, t] = g * M * I
            out["di"][b, t] = g * M * X * I * (1.0 - I)
            out["dr"][b, t] = -rate * dlog * P * (1.0 - P)
            dlam -= scale * _sigmoid(lam) * dlog * P
            g = A * g
        out["dinitial_state"][s] = g
    out["dlam"] = dlam
    out["dr_bias"], out["di_bias"] = out["dr"].sum((0, 1)), out["di"].sum((0, 1))
    return out


def act8(x):
    """The values that x [batch, seqlen, dim] stands for once packed to 8 bits."""
    x = np.asarray(x, dtype=np.float64)
    out = np.zeros_like(x)
    for t in range(0, x.shape[1], GROUP):
        v = x[:, t:t + GROUP]
        top = np.abs(v).max(1, keepdims=True)
        fine = np.isfinite(top)
        _, e = np.frexp(np.where(fine, top, 1.0))
        unit = np.ldexp(1.0, np.where(top == 0.0, -132, np.maximum(e - 1, -126) - 6))
        code = np.clip(np.rint(np.where(fine, v, 0.0) / unit), -127, 127)
        out[:, t:t + GROUP] = np.where(fine, code * unit, np.nan)
    return out


def step(state, x, r, i, lam, r_bias=None, i_bias=None, z=None, slots=None, slots_out=None, scale=8.0):
    """y and the new pool of states."""
    state, x, r, i, lam, r_bias, i_bias, z = _f64(state, x, r, i, lam, r_bias, i_bias, z)
    _, _, iota, a, m = _gates(x, r, i, lam, r_bias, i_bias, scale)
    y, new = np.zeros_like(x), state.copy()
    for b in range(x.shape[0]):
        at = b if slots is None else int(slots[b])
        if not 0 <= at < state.shape[0]:
            continue
        to = at if slots_out is None else int(slots_out[b])
        h = a[b] * state[at] + m[b] * iota[b] * x[b]
        if 0 <= to < state.shape[0]:
            new[to] = h
        y[b] = h if z is None else h * z[b] * _sigmoid(z[b])
    return y, new
