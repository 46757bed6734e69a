"""Plain float64 forms of what stands around the recurrence in a layer -- norm with the
residual's addition, rows in 8-bit integers and their products, short convolution -- for the
tests.  Arrays are numpy; nothing here is shared with the kernels.

The functions that end in _error bound the kernels' float32 arithmetic: the roundings on the
way to each value, each at most U of what it rounds, summed over the formula's terms.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24          # half a unit of float32's last place, relative


def f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def chain(n):
    """Additions that a term of a sum of n passes through: a lane's own, then a tree."""
    return n / 64 + 16


def rms_fwd(s, weight=None, eps=1e-5):
    """y and r [rows, 1] of the rows s as they are kept."""
    s, w = f64(s, weight)
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    y = s * r
    return (y if w is None else y * w), r


def rms_fwd_error(s, weight=None, eps=1e-5):
    """r carries half the sum's error, the division's, the root's (2 units); then two products."""
    y, _ = rms_fwd(s, weight, eps)
    return U * np.abs(y) * (chain(np.shape(s)[-1]) / 2 + 8)


def rms_bwd(s, dy, weight=None, dresidual=None, eps=1e-5):
    s, dy, w, dres = f64(s, dy, weight, dresidual)
    g = dy if w is None else dy * w
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    ds = r * g - s * r ** 3 * (g * s).mean(-1, keepdims=True)
    if dres is not None:
        ds = ds + dres
    return ds, (dy * s * r).reshape(-1, s.shape[-1]).sum(0)


def rms_bwd_error(s, dy, weight=None, dresidual=None, eps=1e-5, depth=None):
    """(of ds, of dweight).  The mean's own error is relative to its terms' magnitudes.  depth: the
    additions that a term of dweight passes through, at most as many as there are rows."""
    s, dy, w, dres = f64(s, dy, weight, dresidual)
    n = chain(s.shape[-1])
    g = dy if w is None else dy * w
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    big = (np.abs(g * s)).mean(-1, keepdims=True)
    ds = U * (np.abs(r * g) * (n / 2 + 8) + np.abs(s) * r ** 3 * big * (2.5 * n + 12))
    if dres is not None:
        ds = ds + U * np.abs(dres)
    terms = np.abs(dy * s * r).reshape(-1, s.shape[-1])
    return ds + U * np.abs(ds), U * terms.sum(0) * ((terms.shape[0] if depth is None else depth) + n / 2 + 8)


def i8_rows(x):
    """(codes, scales) of rows: the scale is a float32 number, the quotients are nearest to the
    real ones.  A row with an infinity or NaN: scale NaN, codes 0."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1, initial=0.0)
    fine = np.isfinite(top)
    scale = np.maximum((np.where(fine, top, 1.0) / 127.0).astype(np.float32), np.float32(2.0 ** -126)).astype(np.float64)
    # a quotient of float32 numbers is at least 2^-33 from a border that it is not on, so one
    # rounding to 53 bits decides nothing
    q = np.rint(np.where(np.isfinite(x), x, 0.0) / scale[..., None])
    return np.where(fine[..., None], q, 0.0).astype(np.int8), np.where(fine, scale, np.nan)


def i8_matmul(a, a_scale, b, b_scale, bias=None):
    a_scale, b_scale, bias = f64(a_scale, b_scale, bias)
    sums = np.asarray(a, np.float64) @ np.asarray(b, np.float64).T     # whole numbers below 2^53
    out = sums * (a_scale[..., None] * b_scale)
    return out if bias is None else out + bias


def i8_matmul_error(a, a_scale, b, b_scale, bias=None):
    """The sum to float32, the product of the scales, theirs, and the addition."""
    out = i8_matmul(a, a_scale, b, b_scale)
    return U * (3.01 * np.abs(out) + (0 if bias is None else np.abs(out + bias)))


def sequences(shape, offsets):
    """(row, begin, end) of every sequence."""
    if offsets is None:
        return [(b, 0, shape[1]) for b in range(shape[0])]
    return [(0, int(lo), int(hi)) for lo, hi in zip(offsets[:-1], offsets[1:])]


def _sigmoid(v):
    w = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + w), w / (1.0 + w))


def _line(x, h0, n, row, lo, hi, dim, K):
    """A sequence's raw inputs with its state in front, [K - 1 + tokens, dim]."""
    start = np.zeros((K - 1, dim)) if h0 is None else h0[n].T
    return np.concatenate([start, x[row, lo:hi]])


def conv_fwd(x, w, b=None, silu=True, initial_state=None, offsets=None):
    """y (zero at padding) and the last states [sequences, dim, K - 1]."""
    x, w, b, h0 = f64(x, w, b, initial_state)
    dim, K = w.shape
    y, last = np.zeros_like(x), []
    for n, (row, lo, hi) in enumerate(sequences(x.shape, offsets)):
        line = _line(x, h0, n, row, lo, hi, dim, K)
        v = sum(line[k:k + hi - lo] * w[:, k] for k in range(K))
        if b is not None:
            v = v + b
        y[row, lo:hi] = v * _sigmoid(v) if silu else v
        last.append(line[hi - lo:].T)
    return y, np.stack(last)


def conv_bwd(x, w, dy, b=None, silu=True, initial_state=None, offsets=None, dlast_state=None, depth=None):
    """Gradients as a dict, and under "error" bounds of the kernels' arithmetic for each.  depth: the
    additions that a term of a parameter's gradient passes through, at most as many as there are tokens."""
    x, w, dy, b, h0, dlast = f64(x, w, dy, b, initial_state, dlast_state)
    dim, K = w.shape
    seqs = sequences(x.shape, offsets)
    out = dict(dx=np.zeros_like(x), dconv_w=np.zeros((dim, K)), dconv_b=np.zeros(dim),
               dinitial_state=np.zeros((len(seqs), dim, K - 1)))
    err = {k: np.zeros_like(v) for k, v in out.items()}
    tokens = x.shape[0] * x.shape[1] + 1 if depth is None else depth
    for n, (row, lo, hi) in enumerate(seqs):
        T = hi - lo
        line = _line(x, h0, n, row, lo, hi, dim, K)
        v = sum(line[k:k + T] * w[:, k] for k in range(K)) + (0 if b is None else b)
        size = sum(np.abs(line[k:k + T] * w[:, k]) for k in range(K)) + (0 if b is None else np.abs(b))
        dv, dve = dy[row, lo:hi].copy(), np.zeros((T, dim))
        if silu:
            g = _sigmoid(v)
            a = np.abs(v)
            slope = g * (1.0 + v * (1.0 - g))
            # g's relative error, through e^-v with the error of its argument, is (|v| + 8) U (1 - g);
            # 1 - g has g's absolute error and a rounding; v's own error moves the slope by half of it
            of_g = (a + 8) * (1 - g)
            e = g * ((1 + a * (1 - g)) * (of_g + 4) + a * (g * of_g + 1)) + 0.5 * (K + 2) * size
            dve = U * np.abs(dv) * (1.2 * e + np.abs(slope))
            dv = dv * slope
        d, de = np.zeros((K - 1 + T, dim)), np.zeros((K - 1 + T, dim))
        if dlast is not None:
            d[T:] += dlast[n].T
            de[T:] += U * np.abs(dlast[n].T)
        for k in range(K):
            d[k:k + T] += w[:, k] * dv
            de[k:k + T] += np.abs(w[:, k]) * (dve + (K + 2) * U * np.abs(dv))
            out["dconv_w"][:, k] += (dv * line[k:k + T]).sum(0)
            err["dconv_w"][:, k] += (np.abs(line[k:k + T]) * (dve + tokens * U * np.abs(dv))).sum(0)
        out["dconv_b"] += dv.sum(0)
        err["dconv_b"] += (dve + tokens * U * np.abs(dv)).sum(0)
        out["dinitial_state"][n], err["dinitial_state"][n] = d[:K - 1].T, de[:K - 1].T
        out["dx"][row, lo:hi], err["dx"][row, lo:hi] = d[K - 1:], de[K - 1:]
    out["error"] = err
    return out


def conv_fwd_error(x, w, b=None, silu=True, initial_state=None, offsets=None):
    x, w, b, h0 = f64(x, w, b, initial_state)
    v, _ = conv_fwd(x, w, b, False, h0, offsets)
    size, _ = conv_fwd(np.abs(x), np.abs(w), None if b is None else np.abs(b), False,
                       None if h0 is None else np.abs(h0), offsets)
    e = (w.shape[1] + 2) * size
    return U * (1.1 * e + np.abs(v * _sigmoid(v)) * (np.abs(v) + 10) if silu else e)


def conv_step(state, x, w, b=None, silu=True, slots=None, slots_out=None):
    """y and the new pool of states."""
    state, x, w, b = f64(state, x, w, b)
    y, new = np.zeros_like(x), state.copy()
    for n in range(x.shape[0]):
        at = n if slots is None else int(slots[n])
        if not 0 <= at < state.shape[0]:
            continue
        to = at if slots_out is None else int(slots_out[n])
        line = np.concatenate([state[at], x[n][:, None]], axis=1)
        v = (line * w).sum(1) + (0 if b is None else b)
        y[n] = v * _sigmoid(v) if silu else v
        if 0 <= to < state.shape[0]:
            new[to] = line[:, 1:]
    return y, new
