"""The float64 forms of the norm, the 8-bit rows and the convolution against autograd, library
routines, rational arithmetic and differences."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import layer

rng = lambda seed: np.random.default_rng(seed)
OFFSETS = [0, 0, 5, 6, 6, 8, 20, 21, 21]


@pytest.mark.parametrize("weighted,added", [(True, True), (False, False), (True, False)])
def test_norm_and_its_gradients_are_autograds(weighted, added):
    r = rng(1)
    x, w, dy, dk = r.normal(size=(6, 33)), r.normal(size=33), r.normal(size=(6, 33)), r.normal(size=(6, 33))
    tx = torch.tensor(x, requires_grad=True)
    tw = torch.tensor(w, requires_grad=True)
    ty = torch.nn.functional.rms_norm(tx, (33,), tw if weighted else None, eps=1e-3)
    loss = (ty * torch.tensor(dy)).sum() + ((tx * torch.tensor(dk)).sum() if added else 0)
    loss.backward()
    y, _ = layer.rms_fwd(x, w if weighted else None, eps=1e-3)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-12)
    ds, dw = layer.rms_bwd(x, dy, w if weighted else None, dk if added else None, eps=1e-3)
    np.testing.assert_allclose(ds, tx.grad.numpy(), rtol=1e-10, atol=1e-13)
    if weighted:
        np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_codes_are_the_nearest_whole_numbers_to_real_quotients():
    r = rng(2)
    x = (r.normal(size=(40, 9)) * np.exp(r.normal(size=(40, 1)) * 20)).astype(np.float32)
    x[0] = 0
    x[1] = np.float32(2.0 ** -140) * r.integers(-100, 100, 9)
    x[2] = [127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5]       # a scale of 1, every one a tie but the first
    codes, scales = layer.i8_rows(x)
    for row, c, s in zip(x, codes, scales):
        assert Fraction(float(s)) >= Fraction(2) ** -126
        for v, q in zip(row, c):
            exact = Fraction(float(v)) / Fraction(float(s))
            assert q == min(127, max(-127, round(exact))), (v, s)     # Python rounds ties to even
    assert codes[2].tolist() == [127, 0, 2, 2, 0, -2, -2, 126, -126]
    bad = np.ones((3, 4))
    bad[0, 1], bad[1, 2] = np.inf, np.nan
    codes, scales = layer.i8_rows(bad)
    assert np.isnan(scales[:2]).all() and not codes[:2].any() and codes[2].tolist() == [127] * 4


def test_products_are_sums_of_whole_numbers():
    r = rng(3)
    a, b = r.integers(-128, 128, (3, 50)), r.integers(-128, 128, (4, 50))
    sa, sb, bias = r.random(3), r.random(4), r.normal(size=4)
    got = layer.i8_matmul(a, sa, b, sb, bias)
    for i in range(3):
        for j in range(4):
            want = Fraction(float(sa[i])) * Fraction(float(sb[j])) * sum(int(p) * int(q) for p, q in zip(a[i], b[j])) \
                + Fraction(float(bias[j]))
            assert abs(got[i, j] - float(want)) < 1e-9


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
def test_convolution_is_the_library_routine(K, silu):
    r = rng(4)
    x, w, b = r.normal(size=(2, 11, 3)), r.normal(size=(3, K)), r.normal(size=3)
    t = torch.nn.functional.conv1d(torch.tensor(x).transpose(1, 2), torch.tensor(w)[:, None], torch.tensor(b), padding=K - 1, groups=3)
    t = t[..., :11].transpose(1, 2)
    want = (torch.nn.functional.silu(t) if silu else t).numpy()
    y, last = layer.conv_fwd(x, w, b, silu)
    np.testing.assert_allclose(y, want, rtol=1e-12, atol=1e-14)
    np.testing.assert_array_equal(last, x[:, 11 - (K - 1):].transpose(0, 2, 1))


def test_convolution_is_the_fused_prologue_of_the_scan():
    r = rng(5)
    x, w, b, h0 = r.normal(size=(2, 9, 5)), r.normal(size=(5, 4)), r.normal(size=5), r.normal(size=(2, 5, 3))
    u, state = oracle.conv_silu_prologue(x, w, b, h0)
    y, last = layer.conv_fwd(x, w, b, True, h0)
    np.testing.assert_allclose(y, u, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(last, state, rtol=0, atol=0)


def test_packed_sequences_are_sequences_by_themselves_and_in_pieces():
    r = rng(6)
    x, w, b, h0 = r.normal(size=(1, 25, 3)), r.normal(size=(3, 4)), r.normal(size=3), r.normal(size=(8, 3, 3))
    y, last = layer.conv_fwd(x, w, b, True, h0, OFFSETS)
    assert not y[0, 21:].any()
    for n, (lo, hi) in enumerate(zip(OFFSETS[:-1], OFFSETS[1:])):
        ys, ls = layer.conv_fwd(x[:, lo:hi], w, b, True, h0[n:n + 1])
        np.testing.assert_allclose(y[:, lo:hi], ys, rtol=0, atol=0)
        np.testing.assert_allclose(last[n:n + 1], ls, rtol=0, atol=0)
        state, pool = h0[n:n + 1], h0[n:n + 1].copy()
        for t in range(lo, hi):                                      # token after token
            yt, pool = layer.conv_step(pool, x[:, t], w, b)
            np.testing.assert_allclose(yt, y[:, t], rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(pool, ls, rtol=0, atol=0)


@pytest.mark.parametrize("offsets,rows", [(None, 2), (OFFSETS, 8)])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [2, 4])
def test_convolution_gradients_by_differences(offsets, rows, silu, K):
    r = rng(7)
    shape = (2, 7, 2) if offsets is None else (1, 25, 2)
    p = dict(x=r.normal(size=shape), w=r.normal(size=(2, K)), b=r.normal(size=2), initial_state=r.normal(size=(rows, 2, K - 1)))
    dy, dlast = r.normal(size=shape), r.normal(size=(rows, 2, K - 1))
    g = layer.conv_bwd(p["x"], p["w"], dy, p["b"], silu, p["initial_state"], offsets, dlast)

    def loss(q):
        y, last = layer.conv_fwd(q["x"], q["w"], q["b"], silu, q["initial_state"], offsets)
        return (y * dy).sum() + (last * dlast).sum()

    for name, grad in (("x", g["dx"]), ("w", g["dconv_w"]), ("b", g["dconv_b"]), ("initial_state", g["dinitial_state"])):
        for at in np.ndindex(p[name].shape):
            e = np.zeros_like(p[name])
            e[at] = 1e-5
            d = (loss({**p, name: p[name] + e}) - loss({**p, name: p[name] - e})) / 2e-5
            assert abs(d - grad[at]) < 1e-8 * (1 + abs(d)), (name, at)


def test_a_row_of_the_pool_that_is_not_used_changes_nothing():
    r = rng(8)
    state, x, w = r.normal(size=(5, 3, 3)), r.normal(size=(3, 3)), r.normal(size=(3, 4))
    y, new = layer.conv_step(state, x, w, slots=[4, -1, 7], slots_out=[0, 1, 2])
    assert not y[1:].any()
    np.testing.assert_array_equal(new[1:], state[1:])
    np.testing.assert_array_equal(new[0], np.concatenate([state[4, :, 1:], x[0][:, None]], 1))


def test_the_norm_before_8_bits_loses_no_more_than_half_a_step():
    r = rng(9)
    y, _ = layer.rms_fwd(r.normal(size=(5, 64)), r.normal(size=64))
    codes, scales = layer.i8_rows(y)
    assert (np.abs(codes * scales[:, None] - y) <= scales[:, None] * (0.5 + 2e-5)).all()


def test_bounds_by_depth_are_below_one_row_or_token():
    """With the additions that a kernel's sums really go through, the bound of a parameter's gradient is
    below the share of one average row of 4094, or token of 26201, so that one left out would show."""
    r = np.random.default_rng(3)
    s, dy, w = r.standard_normal((4094, 40)), r.standard_normal((4094, 40)), r.standard_normal(40)
    _, rr = layer.rms_fwd(s)
    _, bound = layer.rms_bwd_error(s, dy, w, depth=54)
    assert (bound < 0.1 * np.abs(dy * s * rr).mean(0)).all()
    x, dy, w = r.standard_normal((1, 26201, 8)), r.standard_normal((1, 26201, 8)), r.standard_normal((8, 4))
    err = layer.conv_bwd(x, w, dy, silu=False, depth=91)["error"]
    assert (err["dconv_b"] < 0.25 * np.abs(dy).mean((0, 1))).all()
    for k in range(4):
        assert (err["dconv_w"][:, k] < 0.25 * np.abs(dy[0, 3 - k:] * x[0, :26201 - 3 + k]).mean(0)).all()
