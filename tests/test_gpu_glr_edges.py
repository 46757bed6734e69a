"""GPU: the gated linear recurrence and the 8-bit activations where they can go wrong, against
the plain float64 form.  `close` and its bounds are those of the recurrence's
other tests."""
import numpy as np
import pytest
import torch

from oracle import glr
from test_gpu_glr import BF, F32, Work, close, run_fwd, ss  # noqa: F401

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
