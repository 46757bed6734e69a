"""GPU: the gated linear recurrence and the 8-bit activations where they can go wrong, against
the plain float64 form.  `close` and its bounds are those of the recurrence's
other tests."""
import numpy as np
import pytest
import torch

from oracle import glr
from test_gpu_glr import BF, F32, Work, check_bwd, check_fwd, close, run_fwd, ss  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L", [(149, 130), (150, 130), (300, 130), (1, 33000)])
def test_parameter_sums_over_many_tiles(ss, dtype, B, L):  # noqa: F811
    """447 and 450 tiles (around the 448 from which the sums are taken eight tiles at a time),
    900 in short rows, and 516 of one sequence.  Per channel: the sum's terms carry a relative
    error below 3e-6 each, so their sum one below 3e-6 of the sum of their magnitudes; adding
    n of them in partial sums of at most n / 64 adds (n / 64 + 8) 2^-24 of it."""
    w = Work(B, L, 5, dtype, seed=B + L, gate=False)
    _, _, ck = run_fwd(ss, w)
    before = glr.fwd(**w.refs(), **w.par)[2]
    close(ck.view(B, -1, 5), before[:, ::64], F32, "checkpoints")
    dl = torch.from_numpy(w.dl).cuda()
    g = ss.sscan_glr_bwd(dy=w.dy, checkpoints=ck, dlast_state=dl, **w.inputs(), **w.dpar)
    ref = glr.bwd(**w.refs(), dy=w.ref["dy"], dlast_state=w.dl, before=before, **w.par)
    lam = w.par["lam"].astype(np.float64)
    rho = 1 / (1 + np.exp(-(w.ref["r"] + w.par["r_bias"])))
    each = {"dr_bias": ref["dr"], "di_bias": ref["di"],
            "dlam": ref["dr"] / (np.log1p(np.exp(lam)) * (1 + np.exp(-lam)) * (1 - rho))}
    tiles = B * -(-L // 64)
    for k, terms in each.items():
        np.testing.assert_allclose(terms.sum((0, 1)), ref[k], rtol=1e-9, atol=1e-12 * np.abs(terms).sum())
        size = np.abs(terms).sum((0, 1))
        err = np.abs(g[k].double().cpu().numpy() - ref[k])
        assert (err <= (3e-6 + (tiles / 64 + 8) * 2.0 ** -24) * size).all(), (k, err / size)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["r", "i", "x", "lam", "r_bias"])
@pytest.mark.parametrize("offsets", [None, [0, 20, 120, 150]])
def test_nan_reaches_every_gradient_that_depends_on_it(ss, name, dtype, offsets):  # noqa: F811
    """A NaN in one channel: the gradients are not finite exactly where the formula's are not."""
    w = Work(1 if offsets else 2, 150, 8, dtype, seed=9, gate=False, offsets=offsets)
    if name in w.dev:
        w.dev[name][0, 70, 3] = float("nan")
        w.ref[name][0, 70, 3] = np.nan
    else:
        w.dpar[name][3] = float("nan")
        w.par[name][3] = np.nan
    _, _, ck = run_fwd(ss, w)
    g = ss.sscan_glr_bwd(dy=w.dy, checkpoints=ck, dlast_state=torch.from_numpy(w.dl).cuda(), **w.inputs(), **w.dpar)
    ref = glr.bwd(**w.refs(), dy=w.ref["dy"], dlast_state=w.dl, **w.par)
    for k in ("dx", "dr", "di", "dlam", "dr_bias", "di_bias", "dinitial_state"):
        assert np.array_equal(torch.isfinite(g[k]).cpu().numpy(), np.isfinite(ref[k])), k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["x", "r", "i", "z", "dy", "lam"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kept", [False, True])
def test_padding_has_no_gradient_beside_nonfinite_tokens(ss, name, dtype, bad, kept):  # noqa: F811
    """An infinity or NaN in the last request's last tokens, of whose group of 16 the rest is
    padding (or in a parameter): zeros at the padding all the same, and the requests before it,
    whose groups are others, as without it."""
    w = Work(1, 200, 40, dtype, seed=7, offsets=[0, 32, 101])

    def both():
        saved = torch.empty(ss.glr_saved_bytes(1, 200, 40, True), dtype=torch.uint8, device="cuda") if kept else None
        y, _, ck = run_fwd(ss, w, saved=saved)
        given = dict(saved=saved, gated=True) if kept else w.inputs()
        return y, ss.sscan_glr_bwd(dy=w.dy, checkpoints=ck, **given, **w.dpar)

    y0, g0 = both()
    if name == "lam":
        w.dpar["lam"][::3] = bad
    else:
        (w.dy if name == "dy" else w.dev[name])[:, 99, ::3] = bad
    y, g = both()
    assert not y[:, 101:].any()
    for k in ("dx", "dr", "di", "dz"):
        assert not g[k][:, 101:].any(), k              # true of NaN too
        if name != "lam":
            assert torch.equal(g[k][:, :32], g0[k][:, :32]), k
    if name in ("x", "lam", "dy"):                     # it was met (an infinite gate is an open one)
        assert not all(torch.isfinite(g[k][:, 32:101]).all() for k in ("dx", "dr", "di"))


def torch_gates(x, r, i, lam):
    """a, m and the input u in float64, on the GPU (no biases, scale 8)."""
    rate = 8 * torch.nn.functional.softplus(lam.double(), threshold=60)
    q = rate * torch.sigmoid(r.double())
    m = torch.sqrt(-torch.expm1(-2 * q))
    return torch.exp(-q), m, torch.sigmoid(i.double()) * x.double()


def close_there(got, want):
    err = (got.double() - want).abs()
    assert bool((err <= 1e-4 * (1 + want.abs())).all()) and float(err.norm()) <= 3e-6 * float(want.norm())


def test_more_tiles_than_one_grid_row(ss):  # noqa: F811
    """2^24 + 3 sequences of one token and channel, each a workgroup of 256 threads of its own:
    past 2^32 threads, which a launch takes in further rows of its grid only."""
    B = 2 ** 24 + 3
    g = torch.Generator("cuda").manual_seed(1)
    n = lambda: torch.randn(B, 1, 1, generator=g, device="cuda")
    x, r, i, dy = n(), n(), n(), n()
    lam, h0 = torch.tensor([-2.0], device="cuda"), n().view(B, 1)
    ck = torch.empty(ss.glr_checkpoint_bytes(B, 1, 1) // 4, device="cuda")
    y, last = ss.sscan_glr_fwd(x, r, i, lam, initial_state=h0, checkpoints=ck, return_last_state=True)
    a, m, u = torch_gates(x, r, i, lam)
    close_there(y, a * h0.view(B, 1, 1) + m * u)
    assert torch.equal(y.view(B, 1), last) and torch.equal(ck.view(B, 1), h0)
    d = ss.sscan_glr_bwd(lam, dy, ck, x=x, r=r, i=i)
    iota = torch.sigmoid(i.double())
    close_there(d["dx"], dy.double() * m * iota)
    close_there(d["di"], dy.double() * m * u * (1 - iota))
    close_there(d["dinitial_state"], (a * dy.double()).view(B, 1))
    # a sum of 2^24 terms of random sign, by 64 partial sums of 2^18: 2^18 x 2^-24 of the
    # magnitudes at the most, which its roundings' random signs leave far below
    di = dy.double() * m * u * (1 - iota)
    assert abs(float(d["di_bias"][0]) - float(di.sum())) <= 1e-5 * float(di.abs().sum())


def test_more_channels_than_one_grid_row(ss):  # noqa: F811
    """22.5e6 channels: the parameter sums' 12 workgroups of 1024 threads for each 64 of them
    pass 2^32 threads."""
    D = 22_500_001
    g = torch.Generator("cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, r, i, dy = (n(1, 2, D) for _ in range(4))
    lam = n(D) - 2
    ck = torch.empty(ss.glr_checkpoint_bytes(1, 2, D) // 4, device="cuda")
    y = ss.sscan_glr_fwd(x, r, i, lam, checkpoints=ck)
    d = ss.sscan_glr_bwd(lam, dy, ck, x=x, r=r, i=i)
    a, m, u = torch_gates(x, r, i, lam)
    h0 = m[:, 0] * u[:, 0]
    h = torch.stack([h0, a[:, 1] * h0 + m[:, 1] * u[:, 1]], 1)
    close_there(y, h)
    g1 = dy[:, 1].double()
    gs = torch.stack([dy[:, 0].double() + a[:, 1] * g1, g1], 1)
    before = torch.stack([torch.zeros_like(h0), h0], 1)
    dla = gs * (a * before - u * a * a / m)
    rho = torch.sigmoid(r.double())
    want = -8 * torch.sigmoid(lam.double()) * (dla * rho).sum((0, 1))
    size = 8 * torch.sigmoid(lam.double()) * ((gs * a * before).abs() + (gs * u * a * a / m).abs()).sum((0, 1))
    # each term is off by at most 3e-6 of its two parts, the sum by two roundings more
    assert bool(((d["dlam"].double() - want).abs() <= 4e-6 * size).all())
    for k in ("dr", "di"):
        assert torch.allclose(d[k + "_bias"], d[k][0, 0] + d[k][0, 1], rtol=0, atol=0)


def test_more_step_rows_than_one_grid_row(ss):  # noqa: F811
    """2^28 + 5 rows of one channel: past 2^26 workgroups of 64 threads."""
    B = 2 ** 28 + 5
    g = torch.Generator("cuda").manual_seed(3)
    n = lambda: torch.randn(B, 1, generator=g, device="cuda")
    x, r, i, state = n(), n(), n(), n()
    lam, old = torch.tensor([-1.0], device="cuda"), state.clone()
    y = ss.sscan_glr_step(state, x, r, i, lam)
    assert torch.equal(y, state)
    for c in torch.arange(B, device="cuda").split(2 ** 26):
        s = slice(int(c[0]), int(c[-1]) + 1)
        a, m, u = torch_gates(x[s], r[s], i[s], lam)
        close_there(y[s], a * old[s] + m * u)


def test_more_packed_lanes_than_one_grid_row(ss):  # noqa: F811
    """65537 x 65537 single tokens of an odd dim, one lane each: past 2^32 threads.  Whole
    numbers of at most 7 bits are groups of their own here and come back as they were."""
    B = D = 65537
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.empty(B, 1, D, dtype=torch.bfloat16, device="cuda").random_(-127, 128, generator=g)
    packed = ss.sscan_act8_pack(x)
    back = ss.sscan_act8_unpack(packed, (B, 1, D))
    assert torch.equal(back, x)


def test_the_longest_sequence(ss):  # noqa: F811
    """2^30 tokens of one channel, 2^24 tiles in one chain: windows of it against the float64
    form run from 512 tokens before to 512 after, over which the decay, about e^-0.5 a token, leaves
    nothing of what is outside."""
    L = 2 ** 30
    g = torch.Generator("cuda").manual_seed(5)
    x, r, i, dy = (torch.empty(1, L, 1, dtype=BF, device="cuda").normal_(generator=g) for _ in range(4))
    lam = torch.tensor([-2.0], device="cuda")
    ck = torch.empty(ss.glr_checkpoint_bytes(1, L, 1) // 4, device="cuda")
    y, last = ss.sscan_glr_fwd(x, r, i, lam, checkpoints=ck, return_last_state=True)
    d = ss.sscan_glr_bwd(lam, dy, ck, x=x, r=r, i=i)
    for lo in (0, 2 ** 29 - 700, 2 ** 29 + 123456, L - 3000):
        a, b = max(lo - 512, 0), min(lo + 3000 + 512, L)
        cut = lambda t: t[:, a:b].double().cpu().numpy()
        w = dict(x=cut(x), r=cut(r), i=cut(i), lam=np.array([-2.0]))
        ry, rl, _ = glr.fwd(**w)
        rd = glr.bwd(**w, dy=cut(dy))
        inner = slice(lo - a, lo - a + 3000)
        close(y[:, lo:lo + 3000], ry[:, inner], BF, "y")
        for k in ("dx", "dr", "di"):
            close(d[k][:, lo:lo + 3000], rd[k][:, inner], BF, k)
    close(last, rl)
    # the sum of the rounded gradients, 2^-8 of each apart from the sum that was taken
    total, size = (float(f(d["di"]).sum(dtype=torch.float64)) for f in (lambda t: t, torch.abs))
    assert abs(float(d["di_bias"][0]) - total) <= 2.0 ** -8 * size


def test_decay_rates_at_every_size_of_lam(ss):  # noqa: F811
    """One step from a zero state with open gates and x = 1 gives sqrt(1 - a^2), which is about
    the square root of twice the rate: its relative error is half of the rate's, and two units
    of the last place (2^-24) of the square root's own.  The rate goes through about twelve
    roundings or one-ulp functions and 1 - a^2 through six more, each at most 2 x 2^-24 (most
    half of that): below 12 x 2^-24 = 7.2e-7 in all."""
    lam = np.concatenate([np.linspace(-80, -1, 4001), np.linspace(-1, 3, 500)]).astype(np.float32)
    D = lam.size
    f = lambda v: torch.full((1, D), v, device="cuda")
    state = torch.zeros(1, D, device="cuda")
    y = ss.sscan_glr_step(state, f(1.0), f(60.0), f(60.0), torch.from_numpy(lam).cuda())
    rate = 8 * np.log1p(np.exp(lam.astype(np.float64)))
    ref = np.sqrt(-np.expm1(-2 * rate))
    err = np.abs(y.double().cpu().numpy()[0] - ref) / ref
    assert err.max() <= 7.2e-7, (err.max() * 2 ** 24, lam[err.argmax()])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_of_tiny_decay_rates(ss, dtype):  # noqa: F811
    """Rates far below those at which a rounds to 1: the terms with 1 / sqrt(1 - a^2) are the
    formula's, in proportion to each channel's own size."""
    w = Work(2, 140, 24, dtype, seed=10, gate=False)
    lam = np.repeat(np.float32([-75.0, -60.0, -45.0, -30.0, -20.0, -15.0]), 4)
    w.par["lam"], w.dpar["lam"] = lam, torch.from_numpy(lam).cuda()
    _, _, ck = run_fwd(ss, w)
    g = ss.sscan_glr_bwd(dy=w.dy, checkpoints=ck, dlast_state=torch.from_numpy(w.dl).cuda(), **w.inputs(), **w.dpar)
    before = glr.fwd(**w.refs(), **w.par)[2]
    ref = glr.bwd(**w.refs(), dy=w.ref["dy"], dlast_state=w.dl, before=before, **w.par)
    u = 2.0 ** -8 if dtype is BF else 0.0
    for c in range(24):
        for k in ("dx", "dr", "di"):
            got, want = g[k][..., c].double().cpu().numpy(), ref[k][..., c]
            assert np.linalg.norm(got - want) <= (u + 3e-6) * np.linalg.norm(want), (k, lam[c])
    rho = 1 / (1 + np.exp(-(w.ref["r"] + w.par["r_bias"])))
    l64 = lam.astype(np.float64)
    terms = ref["dr"] / (np.log1p(np.exp(l64)) * (1 + np.exp(-l64)) * (1 - rho))
    err = np.abs(g["dlam"].double().cpu().numpy() - ref["dlam"])
    assert (err <= 4e-6 * np.abs(terms).sum((0, 1))).all(), err / np.abs(terms).sum((0, 1))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_8_bit_groups_are_cut_by_position(ss, dtype):  # noqa: F811
    """In 8 bits the 16 tokens of a group share their power of two whatever requests they belong
    to: a NaN takes the tokens of its group with it, those of a neighbour too, and the
    neighbour's gradients that depend on them.  Requests that start at multiples of 16 keep
    apart."""
    def grads(offsets, bad):
        w = Work(1, 96, 5, dtype, seed=3, offsets=offsets)
        if bad is not None:
            w.dev["x"][:, bad] = float("nan")
        saved = torch.empty(ss.glr_saved_bytes(1, 96, 5, True), dtype=torch.uint8, device="cuda")
        y, _, ck = run_fwd(ss, w, saved=saved)
        return y, ss.sscan_glr_bwd(dy=w.dy, checkpoints=ck, saved=saved, gated=True, **w.dpar)

    for offsets, spoilt in (([0, 40, 96], range(32, 48)), ([0, 48, 96], range(0))):
        bad = offsets[1] + 1
        y0, g0 = grads(offsets, None)
        y, g = grads(offsets, bad)
        first = slice(0, offsets[1])
        assert torch.equal(y[:, first], y0[:, first])           # the forward does not read the 8 bits
        gone = torch.isnan(g["di"][0, first]).any(1).cpu().numpy()
        assert np.array_equal(np.flatnonzero(gone), [t for t in spoilt if t < offsets[1]])
        if not len(spoilt):
            assert all(torch.equal(g[k][:, first], g0[k][:, first]) for k in ("dx", "dr", "di", "dz"))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("offsets,L", [([0, 100, 100, 700, 1900], 2000), ([0, 5, 130, 131, 211, 640], 700),
                                       ([0, 16, 64, 128, 129], 300)])
def test_packed_rows_of_whole_cache_lines(ss, dtype, gate, fused, offsets, L):  # noqa: F811
    w = Work(1, L, 128, dtype, seed=6, offsets=offsets, gate=gate, fused=fused)
    ck, before = check_fwd(ss, w)
    check_bwd(ss, w, ck, before)
    n = ss.glr_saved_bytes(1, L, 128, gate)
    saved = torch.full((n,), 77, dtype=torch.uint8, device="cuda")
    run_fwd(ss, w, saved=saved)
    q = {}
    for k, name in enumerate(w.names):
        one = ss.act8_bytes(1, L, 128)
        held = w.ref[name].copy()
        held[:, offsets[-1]:] = 0.0
        q[name] = glr.act8(held)
        v = ss.sscan_act8_unpack(saved[k * one:(k + 1) * one], (1, L, 128), F32)
        assert np.array_equal(v.double().cpu().numpy(), q[name]), name
    q = {k: q.get(k) for k in ("x", "r", "i", "z")}
    check_bwd(ss, w, ck, glr.fwd(**q, **w.par, block_states=before)[2], saved=saved, refs=q)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L", [(2, 77), (1, 1000), (3, 16)])
def test_gated_8_bits_in_whole_cache_lines(ss, dtype, B, L):  # noqa: F811
    w = Work(B, L, 256, dtype, seed=B + L)
    saved = torch.full((ss.glr_saved_bytes(B, L, 256, True),), 77, dtype=torch.uint8, device="cuda")
    _, _, ck = run_fwd(ss, w, saved=saved)
    before = glr.fwd(**w.refs(), **w.par)[2]
    q = {k: glr.act8(v) for k, v in w.refs().items()}
    one = ss.act8_bytes(B, L, 256)
    for k, name in enumerate(w.names):
        v = ss.sscan_act8_unpack(saved[k * one:(k + 1) * one], (B, L, 256), F32)
        assert np.array_equal(v.double().cpu().numpy(), q[name]), name
    check_bwd(ss, w, ck, glr.fwd(**q, **w.par, block_states=before)[2], saved=saved, refs=q)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [70, 33])
def test_packed_requests_over_groups_of_tiles(ss, dtype, D):  # noqa: F811
    w = Work(1, 2500, D, dtype, seed=13, offsets=[0, 100, 100, 700, 700, 701, 1900, 2450])
    check_bwd(ss, w, *check_fwd(ss, w))


def test_a_grid_filled_up_beyond_its_tiles(ss):  # noqa: F811
    """2^22 + 5 sequences of two tiles: 2^23 + 10 workgroups, whose grid of two rows holds nearly
    twice as many; the last states go over the initial ones."""
    B, L = 2 ** 22 + 5, 65
    g = torch.Generator("cuda").manual_seed(6)
    x, r, i, dy = (torch.empty(B, L, 1, device="cuda").normal_(generator=g) for _ in range(4))
    lam = torch.tensor([-3.0], device="cuda")
    state = torch.empty(B, 1, device="cuda").normal_(generator=g)
    h0 = state.double()
    ck = torch.empty(ss.glr_checkpoint_bytes(B, L, 1) // 4, device="cuda")
    y = ss.sscan_glr_fwd(x, r, i, lam, initial_state=state, last_state=state, checkpoints=ck)
    d = ss.sscan_glr_bwd(lam, dy, ck, x=x, r=r, i=i)
    a, m, u = torch_gates(x, r, i, lam)
    h, want = h0, torch.empty_like(a)
    for t in range(L):
        h = a[:, t] * h + m[:, t] * u[:, t]
        want[:, t] = h
    close_there(y, want)
    close_there(state, h)
    e, grad = torch.zeros_like(h), torch.empty_like(a)
    for t in reversed(range(L)):
        grad[:, t] = dy[:, t].double() + e
        e = a[:, t] * grad[:, t]
    close_there(d["dinitial_state"], e)
    close_there(d["dx"], grad * m * torch.sigmoid(i.double()))
