"""The float64 form of the gated linear recurrence and of 8-bit activations, tied to
something other than itself: closed forms, scipy's linear filter, torch's autograd, and
differences of the forward."""
import numpy as np
import pytest

from oracle import glr


def make(B, L, D, seed, gate=True, bias=True, offsets=None, state=True):
    g = np.random.default_rng(seed)
    n = g.standard_normal
    rows = B if offsets is None else len(offsets) - 1
    return dict(x=n((B, L, D)), r=n((B, L, D)), i=n((B, L, D)), lam=g.uniform(-6, 1, D),
                r_bias=n(D) if bias else None, i_bias=n(D) if bias else None, z=n((B, L, D)) if gate else None,
                initial_state=n((rows, D)) if state else None, offsets=offsets, scale=8.0)


def test_constant_decay_is_a_linear_filter():
    from scipy.signal import lfilter
    g = np.random.default_rng(0)
    x, lam = g.standard_normal((1, 200, 3)), np.array([-4.0, -2.0, 0.5])
    r, i = np.full_like(x, 0.3), np.full_like(x, -0.7)
    y, last, _ = glr.fwd(x, r, i, lam, scale=5.0)
    for d in range(3):
        a = np.exp(-5.0 * np.log1p(np.exp(lam[d])) / (1 + np.exp(-0.3)))
        ref = lfilter([np.sqrt(1 - a * a) / (1 + np.exp(0.7))], [1.0, -a], x[0, :, d])
        np.testing.assert_allclose(y[0, :, d], ref, rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(last[0], y[0, -1])


def test_one_token_closed_form():
    w = make(2, 1, 5, 1)
    y, last, before = glr.fwd(**w)
    sig = lambda v: 1 / (1 + np.exp(-v))
    a = np.exp(-8 * np.log(1 + np.exp(w["lam"])) * sig(w["r"][:, 0] + w["r_bias"]))
    h = a * w["initial_state"] + np.sqrt(1 - a * a) * sig(w["i"][:, 0] + w["i_bias"]) * w["x"][:, 0]
    np.testing.assert_allclose(last, h, rtol=1e-9)
    np.testing.assert_allclose(y[:, 0], h * w["z"][:, 0] * sig(w["z"][:, 0]), rtol=1e-9)


def test_steps_equal_the_sequence_and_split_sequences_join():
    w = make(3, 11, 4, 2)
    y, last, _ = glr.fwd(**w)
    state = w["initial_state"].copy()
    for t in range(11):
        yt, state = glr.step(state, w["x"][:, t], w["r"][:, t], w["i"][:, t], w["lam"], w["r_bias"], w["i_bias"],
                             w["z"][:, t])
        np.testing.assert_allclose(yt, y[:, t], rtol=1e-12)
    np.testing.assert_allclose(state, last, rtol=1e-12)


def test_packed_equals_each_request_alone():
    off = np.array([0, 0, 3, 4, 4, 90, 90], np.int32)
    w = make(1, 95, 3, 3, offsets=off)
    y, last, _ = glr.fwd(**w)
    dy = np.random.default_rng(4).standard_normal(w["x"].shape)
    dl = np.random.default_rng(5).standard_normal(last.shape)
    g = glr.bwd(dy=dy, dlast_state=dl, **w)
    total = 0.0
    for s in range(6):
        c = slice(off[s], off[s + 1])
        one = {k: (v[:, c] if k in ("x", "r", "i", "z") else v) for k, v in w.items()}
        one.update(offsets=None, initial_state=w["initial_state"][s:s + 1])
        ys, ls, _ = glr.fwd(**one)
        np.testing.assert_allclose(y[:, c], ys)
        np.testing.assert_allclose(last[s], ls[0])
        gs = glr.bwd(dy=dy[:, c], dlast_state=dl[s:s + 1], **one)
        for k in ("dx", "dr", "di", "dz"):
            np.testing.assert_allclose(g[k][:, c], gs[k])
        np.testing.assert_allclose(g["dinitial_state"][s], gs["dinitial_state"][0])
        total = total + gs["dlam"]
    np.testing.assert_allclose(g["dlam"], total)
    assert not y[:, 90:].any() and not g["dx"][:, 90:].any()


@pytest.mark.parametrize("gate,offsets", [(True, None), (False, None), (True, [0, 4, 4, 9])])
def test_gradients_by_differences(gate, offsets):
    """Central differences with step e: truncation ~ e^2 |f'''| ~ 1e-10, rounding ~ 1e-15 / e
    ~ 1e-10, so 1e-7 relative to the largest gradient leaves a wide margin."""
    off = None if offsets is None else np.array(offsets, np.int32)
    w = make(1 if off is not None else 2, 10, 3, 6, gate=gate, offsets=off)
    g = np.random.default_rng(7)
    y, last, _ = glr.fwd(**w)
    dy, dl = g.standard_normal(y.shape), g.standard_normal(last.shape)
    loss = lambda q: (glr.fwd(**q)[0] * dy).sum() + (glr.fwd(**q)[1] * dl).sum()
    got = glr.bwd(dy=dy, dlast_state=dl, **w)
    names = dict(x="dx", r="dr", i="di", lam="dlam", r_bias="dr_bias", i_bias="di_bias",
                 initial_state="dinitial_state", **({"z": "dz"} if gate else {}))
    e = 1e-5
    for k, gk in names.items():
        ref = np.zeros_like(w[k])
        for at in np.ndindex(w[k].shape):
            both = []
            for sign in (1, -1):
                q = dict(w)
                q[k] = w[k].copy()
                q[k][at] += sign * e
                both.append(loss(q))
            ref[at] = (both[0] - both[1]) / (2 * e)
        assert np.abs(got[gk] - ref).max() <= 1e-7 * (1 + np.abs(ref).max()), k


def test_gradients_by_autograd():
    import torch
    w = make(2, 23, 4, 8)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in w.items() if isinstance(v, np.ndarray)}
    rho, iota = torch.sigmoid(t["r"] + t["r_bias"]), torch.sigmoid(t["i"] + t["i_bias"])
    a = torch.exp(-8.0 * torch.nn.functional.softplus(t["lam"], threshold=100) * rho)
    h, ys = t["initial_state"], []
    for k in range(23):
        h = a[:, k] * h + torch.sqrt(1 - a[:, k] ** 2) * iota[:, k] * t["x"][:, k]
        ys.append(h * torch.nn.functional.silu(t["z"][:, k]))
    dy = np.random.default_rng(9).standard_normal((2, 23, 4))
    (torch.stack(ys, 1) * torch.tensor(dy)).sum().backward()
    got = glr.bwd(dy=dy, **w)
    for k, gk in dict(x="dx", r="dr", i="di", z="dz", lam="dlam", r_bias="dr_bias", i_bias="di_bias",
                      initial_state="dinitial_state").items():
        np.testing.assert_allclose(got[gk], t[k].grad.numpy(), rtol=1e-8, atol=1e-11, err_msg=k)


def test_act8_properties():
    g = np.random.default_rng(10)
    x = (g.standard_normal((2, 37, 5)) * np.exp(3 * g.standard_normal(5))).astype(np.float32).astype(np.float64)
    q = glr.act8(x)
    for t in range(0, 37, 16):
        v, w = x[:, t:t + 16], q[:, t:t + 16]
        e = np.floor(np.log2(np.abs(v).max(1, keepdims=True)))
        # whole multiples of 2^(e-6), at most 127 of them, each within half a unit of the
        # value unless its nearest multiple was 128
        c = w / 2.0 ** (e - 6)
        assert (c == np.rint(c)).all() and np.abs(c).max() <= 127
        err = np.abs(v - w) / 2.0 ** (e - 6)
        assert err.max() < 1 and (err[np.abs(c) < 127] <= 0.5).all()
    np.testing.assert_array_equal(glr.act8(q), q)            # packed values stay
    assert not glr.act8(np.zeros((1, 20, 2))).any()
    tiny = np.full((1, 16, 1), 2.0 ** -140)                  # below the smallest exponent kept
    assert np.abs(glr.act8(tiny) - tiny).max() <= 2.0 ** -133
    bad = x.copy()
    bad[0, 20, 1] = np.inf
    out = glr.act8(bad)
    assert np.isnan(out[0, 16:32, 1]).all() and np.isfinite(np.delete(out[0], 1, axis=1)).all()
