"""The norm, the 8-bit rows and products and the convolution as they are used: one after another
around the recurrence in training and in decoding, in captured graphs, on streams of their own, on
tensors past 32 bits of elements, for many requests, and in the example's model."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import glr, layer
from test_gpu_layer import BF16, F32, HALF, close, dev, host, normal, same, ss  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECURRENCE = 1e-4        # what the gated recurrence's float32 results are held to, of 1 + their size


def indices(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------
# One after another
# ---------------------------------------------------------------------------------------

class Layer:
    """Norm, convolution of the normed tokens, and the recurrence on them, packed, in float32."""

    def __init__(self, tokens=203, dim=36, offsets=(0, 0, 64, 67, 190)):
        n = lambda k, *s: normal(k, *s)
        self.off = np.array(offsets, np.int32)
        self.doff = torch.from_numpy(self.off).cuda()
        self.u, self.res, self.weight = n(1, 1, tokens, dim), n(2, 1, tokens, dim), n(3, dim)
        self.conv_w, self.conv_b = n(4, dim, 4) * 0.3, n(5, dim)
        self.r, self.i, self.lam = n(6, 1, tokens, dim), n(7, 1, tokens, dim), n(8, dim) - 3
        self.dy, self.dres = n(9, 1, tokens, dim), n(10, 1, tokens, dim)
        self.rows = len(offsets) - 1

    def forward(self, ss, u):
        v = ss.sscan_rms_fwd(u, self.weight, residual=self.res)
        x = ss.sscan_dwconv_fwd(v["y"], self.conv_w, self.conv_b, offsets=self.doff)
        ck = torch.empty(ss.glr_checkpoint_bytes(*u.shape) // 4, device="cuda")
        y = ss.sscan_glr_fwd(x, self.r, self.i, self.lam, offsets=self.doff, checkpoints=ck)
        return v, x, ck, y

    def backward(self, ss, v, x, ck):
        g = ss.sscan_glr_bwd(self.lam, self.dy, ck, x=x, r=self.r, i=self.i, offsets=self.doff)
        c = ss.sscan_dwconv_bwd(v["y"], self.conv_w, g["dx"], self.conv_b, offsets=self.doff)
        n = ss.sscan_rms_bwd(v["residual"], self.weight, c["dx"], dresidual=self.dres)
        return g, c, n

    def oracle(self, u):
        """The same in 64 bits: (y, gradients of u, conv_w, conv_b and weight)."""
        w, cw, cb, lam = (host(t) for t in (self.weight, self.conv_w, self.conv_b, self.lam))
        r, i, dy = host(self.r), host(self.i), host(self.dy)
        s = u + host(self.res)
        v, _ = layer.rms_fwd(s, w)
        x, _ = layer.conv_fwd(v, cw, cb, offsets=self.off)
        y, _, before = glr.fwd(x, r, i, lam, offsets=self.off)
        g = glr.bwd(x, r, i, lam, dy, offsets=self.off, before=before)
        c = layer.conv_bwd(v, cw, g["dx"], cb, offsets=self.off)
        ds, dw = layer.rms_bwd(s, c["dx"], w, host(self.dres))
        return y, dict(u=ds, conv_w=c["dconv_w"], conv_b=c["dconv_b"], weight=dw)


def test_a_layer_and_its_gradients(ss):  # noqa: F811
    """Against the same layer in 64 bits.  The recurrence's gradient is off by RECURRENCE; the
    convolution passes that on at most times 1.1 sum |conv_w| (1.1 bounds silu's slope), the norm
    times |weight| r and once more by way of the mean; sums over tokens add up."""
    w = Layer()
    v, x, ck, y = w.forward(ss, w.u)
    g, c, n = w.backward(ss, v, x, ck)
    want, grads = w.oracle(host(w.u))
    assert np.abs(host(y) - want).max() <= RECURRENCE * (1 + np.abs(want).max())
    taps = 1.1 * np.abs(host(w.conv_w)).sum(1).max()
    _, r = layer.rms_fwd(host(w.u) + host(w.res), host(w.weight))
    size = RECURRENCE * (1 + np.abs(host(g["dx"])).max())
    through = size * taps * np.abs(host(w.weight)).max() * r.max()
    assert np.abs(host(n["dx"]) - grads["u"]).max() <= through * (1 + 36 ** 0.5)
    tokens = w.u.shape[1]
    for got, name in ((c["dconv_w"], "conv_w"), (c["dconv_b"], "conv_b"), (n["dweight"], "weight")):
        assert np.abs(host(got) - grads[name]).max() <= RECURRENCE * (1 + np.abs(grads[name]).max()) * max(1, taps), name
    assert tokens > w.off[-1] and not host(c["dx"])[0, w.off[-1]:].any()


def test_a_layers_gradient_by_differences(ss):  # noqa: F811
    """Central differences along a direction, with a step of 2^-6: the truncation is e^2 / 6 of the
    third derivative, which along a direction of size 1 an element is below 10 of the first for
    these smooth functions; rounding, 2^-24 of sums of some 7000 terms over e, is far below it."""
    w = Layer()
    v, x, ck, y = w.forward(ss, w.u)
    _, _, n = w.backward(ss, v, x, ck)
    step = normal(20, *w.u.shape)
    e = 2.0 ** -6

    def loss(u):
        v, _, _, y = w.forward(ss, u)
        inside = slice(0, int(w.off[-1]))
        return float((y[:, inside].double() * w.dy[:, inside].double()).sum() + (v["residual"].double() * w.dres.double()).sum())

    slope = (loss(w.u + e * step) - loss(w.u - e * step)) / (2 * e)
    whole = float((n["dx"].double() * step.double()).sum())
    size = float((n["dx"].double() * step.double()).square().sum().sqrt())
    assert abs(slope - whole) <= e * e / 6 * 10 * size + 1e-3 * size


def test_a_layer_decodes_in_8_bits(ss):  # noqa: F811
    """One token for a batch with an idle row, each operator held to its float64 form at what it was
    given, in bfloat16 with a float32 stream; then again from the states that it left."""
    batch, width, dim = 5, 72, 40
    slots = indices(3, 0, -1, 6, 2)
    inward, outward = (ss.sscan_i8_quant(normal(k, *s, dtype=BF16)) for k, s in ((1, (2 * dim, width)), (2, (width, dim))))
    norm, cw, cb, lam = normal(3, width), normal(4, dim, 4), normal(5, dim), normal(6, dim) - 3
    conv, state, stream = normal(7, 8, dim, 3), normal(8, 8, dim), normal(9, batch, width)
    u = normal(10, batch, width, dtype=BF16)
    gate = normal(11, batch, dim, dtype=BF16)
    for _ in range(3):
        v = ss.sscan_rms_fwd(u, norm, residual=stream, want_codes=True)
        s = (u.float() + stream).double().cpu().numpy()
        close(v["residual"], s, 2.0 ** -24 * np.abs(s), "stream")
        y, _ = layer.rms_fwd(host(v["residual"]), host(norm))
        err = layer.rms_fwd_error(host(v["residual"]), host(norm))
        scales = host(v["scales"])[:, None]
        assert (np.abs(host(v["codes"]) * scales - y) <= 0.5 * scales + err + scales * 127 * 2.0 ** -23).all()
        p = ss.sscan_i8_matmul(v["codes"], v["scales"], *inward)
        args = (host(v["codes"]), host(v["scales"]), host(inward[0]), host(inward[1]))
        close(p, layer.i8_matmul(*args), layer.i8_matmul_error(*args), "inward")
        x, r = p.split(dim, dim=1)
        before, held = host(conv), host(state)
        xc = ss.sscan_dwconv_step(conv, x, cw, cb, slots=slots)
        want, after = layer.conv_step(before, host(x), host(cw), host(cb), slots=host(slots))
        close(xc, want, 2.0 ** -20 * (1 + np.abs(want)), "convolution")
        np.testing.assert_array_equal(host(conv), after)
        h = ss.sscan_glr_step(state, xc, r, gate, lam, slots=slots)
        want, after = glr.step(held, host(xc), host(r), host(gate), host(lam), slots=host(slots).astype(int))
        close(h, want, RECURRENCE * (1 + np.abs(want)), "recurrence")
        assert np.abs(host(state) - after).max() <= RECURRENCE * (1 + np.abs(after).max())
        codes, scales = ss.sscan_i8_quant(h)
        wc, ws = layer.i8_rows(host(h))
        np.testing.assert_array_equal(host(codes), wc)
        np.testing.assert_array_equal(host(scales), ws)
        u = ss.sscan_i8_matmul(codes, scales, *outward)
        args = (wc, ws, host(outward[0]), host(outward[1]))
        close(u, layer.i8_matmul(*args), layer.i8_matmul_error(*args), "outward")
        assert not host(u)[2].any()          # the idle row's recurrence gives 0
        stream = v["residual"]


# ---------------------------------------------------------------------------------------
# Graphs, streams
# ---------------------------------------------------------------------------------------

class Calls:
    """Every operator once on inputs of its own, results in `out` if given."""

    def __init__(self, ss, seed, rows=700, dim=264, dtype=BF16):
        self.ss, n = ss, lambda k, *s: normal(seed + k, *s, dtype=dtype)
        self.x, self.res, self.dy = n(1, 1, rows, dim), n(2, 1, rows, dim), n(3, 1, rows, dim)
        self.w, self.conv_w, self.conv_b = normal(seed + 4, dim), normal(seed + 5, dim, 4), normal(seed + 6, dim)
        self.codes = ss.sscan_i8_quant(n(7, 300, dim))
        self.off = indices(0, 5, rows // 2, rows - 3)
        self.h0, self.pool = normal(seed + 8, 3, dim, 3), normal(seed + 9, 9, dim, 3)
        self.slots = indices(4, -1, 0)
        self.work = torch.empty(max(ss.rms_bwd_workspace_size(rows, dim), ss.dwconv_bwd_workspace_size(1, rows, dim, 4)),
                                dtype=torch.uint8, device="cuda")

    def __call__(self, out=None, work=None):
        ss, out = self.ss, out if out is not None else {}
        get = lambda k: out.get(k)
        a = ss.sscan_rms_fwd(self.x, self.w, residual=self.res, want_codes=True, out=get("norm"))
        b = ss.sscan_i8_matmul(a["codes"], a["scales"], *self.codes, out=get("product"))
        few = ss.sscan_i8_matmul(a["codes"][0, :3], a["scales"][0, :3], *self.codes, out=get("few"))
        c = ss.sscan_dwconv_fwd(a["y"], self.conv_w, self.conv_b, initial_state=self.h0, offsets=self.off, out=get("conv"))
        g = ss.sscan_dwconv_bwd(a["y"], self.conv_w, self.dy, self.conv_b, initial_state=self.h0, offsets=self.off,
                                out=get("dconv"), workspace=work)
        d = ss.sscan_rms_bwd(a["residual"], self.w, g["dx"], dresidual=self.dy, out=get("dnorm"), workspace=work)
        q = ss.sscan_i8_quant(c)
        pool = self.pool.clone()
        s = ss.sscan_dwconv_step(pool, self.x[0, :3], self.conv_w, self.conv_b, slots=self.slots)
        return dict(norm=a, product=b, few=few, conv=c, dconv=g, dnorm=d, quant=dict(c=q[0], s=q[1]), step=dict(y=s, pool=pool))


def flat(r):
    return {(k, n): t for k, v in r.items() for n, t in (v.items() if isinstance(v, dict) else [("", v)])}


def equal(got, want, name):
    got, want = flat(got), flat(want)
    assert set(got) == set(want)
    for k in want:
        same(got[k], want[k], f"{name} {k}")


def test_graph_replays(ss):  # noqa: F811
    """Captured once with its own buffers, replayed on changing inputs between eager calls."""
    c = Calls(ss, 30)
    c(work=c.work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = c(work=c.work)
    for k in range(4):
        c.x.add_(0.25)
        c.dy.mul_(1.125)
        graph.replay()
        torch.cuda.synchronize()
        equal(held, c(), f"replay {k}")
        torch.cuda.synchronize()


def test_two_graphs_with_one_workspace(ss):  # noqa: F811
    """Replayed one after the other on a stream: each has its sums joined before the next begins."""
    pair = [Calls(ss, 40), Calls(ss, 60, rows=900)]
    work = pair[1].work if pair[1].work.numel() >= pair[0].work.numel() else pair[0].work
    for c in pair:
        c(work=work)
    torch.cuda.synchronize()
    graphs, held = [], []
    for c in pair:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(c(work=work))
    for k in range(3):
        for c in pair:
            c.x.mul_(1.0625)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for c, h in zip(pair, held):
            equal(h, c(), f"replay {k}")


def test_two_streams_at_once(ss):  # noqa: F811
    pair = [Calls(ss, 70, rows=3000, dim=520), Calls(ss, 90, rows=2000, dim=1100, dtype=F32)]
    alone = [c() for c in pair]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(4):
        for k, c in enumerate(pair):
            with torch.cuda.stream(streams[k]):
                got[k].append(c())
    torch.cuda.synchronize()
    for k in range(2):
        for n, r in enumerate(got[k]):
            equal(r, alone[k], f"stream {k}, call {n}")


def test_results_into_given_tensors(ss):  # noqa: F811
    c = Calls(ss, 50)
    want = c()
    out = {k: {n: torch.full_like(t, 5) for n, t in v.items()} if isinstance(v, dict) else torch.full_like(v, 5)
           for k, v in want.items()}
    equal(c(out=out), want, "given")
    for k, t in flat(out).items():
        if k[0] not in ("quant", "step"):
            same(t, flat(want)[k], str(k))


# ---------------------------------------------------------------------------------------
# Large and many
# ---------------------------------------------------------------------------------------

def filled(*shape, seed, dtype=BF16):
    """Normal values, a slice of the first dimension at a time."""
    g = torch.Generator("cuda").manual_seed(seed)
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    for k in range(0, shape[0], max(1, shape[0] // 8)):
        t[k:k + max(1, shape[0] // 8)].normal_(generator=g)
    return t


def test_norm_past_32_bits(ss):  # noqa: F811
    rows, dim = 70000, 32768                       # 2.29e9 elements
    x, w = filled(rows, dim, seed=1), normal(2, dim)
    at = [0, 32767, 65535, 65536, rows - 1]
    out = ss.sscan_rms_fwd(x, w, want_codes=True)
    y, _ = layer.rms_fwd(host(x[at]), host(w))
    err = layer.rms_fwd_error(host(x[at]), host(w))
    close(out["y"][at], y, err, "y")
    scales = host(out["scales"][at])[:, None]
    assert (np.abs(host(out["codes"][at]) * scales - y) <= 0.5 * scales + err + scales * 127 * 2.0 ** -23).all()
    assert bool(out["y"][-100:].isfinite().all())
    q, s = ss.sscan_i8_quant(x)
    wq, ws = layer.i8_rows(host(x[at]))
    np.testing.assert_array_equal(host(q[at]), wq)
    np.testing.assert_array_equal(host(s[at]), ws)
    del q, out
    dx = ss.sscan_rms_bwd(x, w, x, want_dweight=False)["dx"]
    ds, _ = layer.rms_bwd(host(x[at]), host(x[at]), host(w))
    close(dx[at], ds, layer.rms_bwd_error(host(x[at]), host(x[at]), host(w))[0], "dx")


def test_products_past_32_bits(ss):  # noqa: F811
    """Outputs past 2^31, a side's rows past 2^31 bytes, and rows 2^23 bytes apart and more."""
    def check(a, sa, b, sb, rows):
        got = ss.sscan_i8_matmul(a, sa, b, sb)
        assert bool(got.isfinite().all())
        args = (host(a[rows]), host(sa[rows]), host(b), host(sb))
        close(got[rows], layer.i8_matmul(*args), layer.i8_matmul_error(*args), "product")

    g = torch.Generator("cuda").manual_seed(3)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)
    ones = lambda n, k: normal(k, n).abs() + 0.1
    m, n, k = 70000, 32768, 128
    check(codes(m, k), ones(m, 1), codes(n, k), ones(n, 2), [0, 65535, 65536, m - 1])
    wide = torch.empty(m, 40000, dtype=torch.int8, device="cuda")
    for start in (0, 39000, 39856):
        a = wide[:, start:start + 144]
        a.copy_(codes(m, 144))
        check(a, ones(m, 3), codes(200, 144), ones(200, 4), [0, 53687, m - 1])
        a = wide[:, start:start + 128]
        check(a, ones(m, 3), codes(200, 128), ones(200, 4), [0, 53687, m - 1])
    del wide
    wide = torch.empty(300, (1 << 23) + 16, dtype=torch.int8, device="cuda")
    a = wide[:, 5 << 20:(5 << 20) + 256]
    a.copy_(codes(300, 256))
    check(a, ones(300, 5), codes(130, 256), ones(130, 6), [0, 150, 299])
    check(codes(130, 256), ones(130, 6), a, ones(300, 5), [0, 129])
    check(a[:7], ones(7, 5), codes(130, 256), ones(130, 6), [0, 6])


def test_products_of_the_most_rows(ss):  # noqa: F811
    """2^31 - 1 rows of either side: the last tile would reach past what 31 bits count."""
    most, k = 2 ** 31 - 1, 16
    g = torch.Generator("cuda").manual_seed(4)
    codes = lambda n: torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    many, scales = torch.zeros(most, k, dtype=torch.int8, device="cuda"), torch.ones(most, device="cuda")
    few, fs = codes(17), normal(1, 17).abs() + 0.1
    for at in (0, 2 ** 30, most - 300):
        many[at:at + 300] = codes(300)
        scales[at:at + 300] = normal(2, 300).abs() + 0.1
    for turn, n in ((0, 17), (1, 17), (0, 1)):
        a, sa, b, sb = (few[:n], fs[:n], many, scales) if turn == 0 else (many, scales, few[:n], fs[:n])
        out = ss.sscan_i8_matmul(a, sa, b, sb)
        for at in (0, 2 ** 30, most - 300):
            part = slice(at, at + 300)
            if turn == 0:
                args, got = (host(a), host(sa), host(b[part]), host(sb[part])), out[:, part]
            else:
                args, got = (host(a[part]), host(sa[part]), host(b), host(sb)), out[part]
            close(got, layer.i8_matmul(*args), layer.i8_matmul_error(*args), f"rows from {at}")
        rest = out[:, 300:2 ** 30] if turn == 0 else out[300:2 ** 30]
        assert not bool(rest[..., :4096].any()) and not bool((rest[:, -4096:] if turn == 0 else rest[-4096:]).any())
        del out, rest


def test_convolution_past_32_bits(ss):  # noqa: F811
    L, D = (1 << 20) + 5, 2304                     # 2.4e9 elements in one row
    x, dy = filled(L, D, seed=1)[None], filled(L, D, seed=2)[None]
    w, b = normal(3, D, 4), normal(4, D)
    cut = 1000003
    off = indices(0, 17, cut, L - 2)
    y, last = ss.sscan_dwconv_fwd(x, w, b, offsets=off, return_last_state=True)
    g = ss.sscan_dwconv_bwd(x, w, dy, b, offsets=off)
    cols = [0, 1000, D - 1]
    for lo, hi, first in ((0, 17, 0), (cut, L - 2, 0), (cut - 400, cut, 3)):
        pick = lambda t: host(t[:, lo:hi][:, :, cols])
        args = (pick(x), host(w[cols]), host(b[cols]))
        want, _ = layer.conv_fwd(*args)
        err = layer.conv_fwd_error(*args)
        close(y[:, lo + first:hi][:, :, cols], want[:, first:], err[:, first:], "y")
        r = layer.conv_bwd(*args[:2], pick(dy), args[2])
        close(g["dx"][:, lo + first:hi][:, :, cols], r["dx"][:, first:], r["error"]["dx"][:, first:], "dx")
    assert not bool(y[0, L - 2:].any()) and not bool(g["dx"][0, L - 2:].any())
    same(last[2], x[0, L - 5:L - 2].t().float(), "last state")
    assert bool(g["dconv_w"].isfinite().all())


def test_convolution_step_in_a_large_pool(ss):  # noqa: F811
    slots, dim = 200000, 4096                      # 2.46e9 elements
    pool = torch.zeros(slots, dim, 3, device="cuda")
    x, w = normal(1, 4, dim, dtype=BF16), normal(2, dim, 4)
    at = indices(slots - 1, 5, 174763, -1)
    h0 = normal(3, 3, dim, 3)
    pool[at[:3].long()] = h0
    y = ss.sscan_dwconv_step(pool, x, w, slots=at)
    want, after = layer.conv_step(host(h0), host(x), host(w), slots=[0, 1, 2, -1])
    close(y, want, 2.0 ** -20 * (1 + np.abs(want)), "y")
    np.testing.assert_array_equal(host(pool[at[:3].long()]), after)
    pool[at[:3].long()] = 0
    assert not bool(pool.any())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_convolution_of_many_requests(ss, dtype):  # noqa: F811
    """A thousand requests of 0 to 40 tokens with carried states, forward and backward."""
    g = np.random.default_rng(8)
    off = np.concatenate([[0], np.cumsum(g.integers(0, 41, 1000))]).astype(np.int32)
    L, D = int(off[-1]) + 13, 68
    x, dy = normal(1, 1, L, D, dtype=dtype), normal(2, 1, L, D, dtype=dtype)
    w, b, h0, dlast = normal(3, D, 4), normal(4, D), normal(5, 1000, D, 3), normal(6, 1000, D, 3)
    doff = torch.from_numpy(off).cuda()
    y, last = ss.sscan_dwconv_fwd(x, w, b, initial_state=h0, offsets=doff, return_last_state=True)
    args = (host(x), host(w), host(b), True, host(h0), off)
    want, wlast = layer.conv_fwd(*args)
    close(y, want, layer.conv_fwd_error(*args), "y")
    np.testing.assert_array_equal(host(last), wlast)
    got = ss.sscan_dwconv_bwd(x, w, dy, b, initial_state=h0, offsets=doff, dlast_state=dlast)
    r = layer.conv_bwd(host(x), host(w), host(dy), host(b), True, host(h0), off, host(dlast))
    for k in ("dx", "dconv_w", "dconv_b", "dinitial_state"):
        close(got[k], r[k], r["error"][k], k)


# ---------------------------------------------------------------------------------------
# The example's model
# ---------------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("block", os.path.join(ROOT, "examples", "gated_recurrence_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_norm_gradients(block):
    u, res = normal(1, 1, 50, 40, dtype=BF16).requires_grad_(), normal(2, 1, 50, 40).requires_grad_()
    w = normal(3, 40).requires_grad_()
    dy, ds = normal(4, 1, 50, 40, dtype=BF16), normal(5, 1, 50, 40)
    y, s = block.Norm.apply(u, res, w)
    torch.autograd.backward([y, s], [dy, ds])
    want, dw = layer.rms_bwd(host(s), host(dy), host(w), host(ds))
    eds, edw = layer.rms_bwd_error(host(s), host(dy), host(w), host(ds))
    close(u.grad, want, eds, "u")
    close(res.grad, want, eds, "residual")
    close(w.grad, dw, edw, "weight")


def test_example_recurrence_gradients(block, ss):  # noqa: F811
    """Of the product's columns and the parameters, against the float64 forms in the same order; the
    recurrence's backward takes its inputs in 8 bits, and starts each block from the kept state."""
    tokens, dim, off = 150, 20, np.array([0, 0, 70, 71, 141], np.int32)
    p = normal(1, 1, tokens, 4 * dim).requires_grad_()
    cw, cb, lam, rb, ib = (t.requires_grad_() for t in (normal(2, dim, 4) * 0.3, normal(3, dim), normal(4, dim) - 3, normal(5, dim),
                                                        normal(6, dim)))
    dy = normal(7, 1, tokens, dim)
    y = block.GatedRecurrence.apply(p, cw, cb, lam, rb, ib, torch.from_numpy(off).cuda())
    y.backward(dy)
    x, r, i, z = np.split(host(p), 4, axis=2)
    xc, _ = layer.conv_fwd(x, host(cw), host(cb), offsets=off)
    par = dict(lam=host(lam), r_bias=host(rb), i_bias=host(ib), offsets=off)
    want, _, before = glr.fwd(xc, r, i, z=z, **par)
    assert np.abs(host(y) - want).max() <= RECURRENCE * (1 + np.abs(want).max())
    # what 8 bits keep is taken from the float32 values: a value next to a border may fall either way
    xk = ss.sscan_dwconv_fwd(p.detach()[..., :dim], cw.detach(), cb.detach(), offsets=torch.from_numpy(off).cuda())
    used = np.arange(tokens)[:, None] < off[-1]             # padding does not count for a group's scale
    q = {k: glr.act8(v * used) for k, v in dict(x=host(xk), r=r, i=i, z=z).items()}
    g = glr.bwd(**q, dy=host(dy), **par, before=glr.fwd(**q, **par, block_states=before)[2])
    c = layer.conv_bwd(x, host(cw), g["dx"], host(cb), offsets=off)
    taps = max(1.0, 1.1 * np.abs(host(cw)).sum(1).max())
    for got, ref in ((p.grad, np.concatenate([c["dx"], g["dr"], g["di"], g["dz"]], 2)), (cw.grad, c["dconv_w"]), (cb.grad, c["dconv_b"]),
                     (lam.grad, g["dlam"]), (rb.grad, g["dr_bias"]), (ib.grad, g["di_bias"])):
        assert np.abs(host(got) - ref).max() <= RECURRENCE * (1 + np.abs(ref).max()) * taps


def test_example_serves_prefill_and_decode_alike(block):
    """Three layers, requests of one token among others: a decoded token's states and codes are those
    of the prefill up to rounding that differs by half a step of bfloat16 in a layer's outputs."""
    torch.manual_seed(3)
    first, last, worst = block.main(steps=2, depth=3, tell=lambda *a: None)
    assert np.isfinite([first, last]).all() and worst <= 0.05


def test_convolution_past_many_empty_requests(ss):  # noqa: F811
    """A million empty requests between two others: the second is found at once, wherever a block of
    tokens meets it.  With the empty ones in front, which the search at a block's first token passes,
    the same calls take some 0.1 ms; one after another the empty ones took 80 ns each, 84 ms a pass."""
    L, D, many = 200, 72, 1 << 20
    x, dy, w, b = normal(1, 1, L, D), normal(2, 1, L, D), normal(3, D, 4), normal(4, D)
    two = torch.tensor([0, 103, 190], dtype=torch.int32, device="cuda")
    fill = lambda v: torch.full((many,), v, dtype=torch.int32, device="cuda")
    middle, front = torch.cat([two[:2], fill(103), two[2:]]), torch.cat([fill(0), two])

    def both(off):
        y = ss.sscan_dwconv_fwd(x, w, b, offsets=off)
        return y, ss.sscan_dwconv_bwd(x, w, dy, b, offsets=off, want_dinitial_state=False)

    want = both(two)
    took = []
    for off in (middle, front):
        y, g = both(off)
        same(y, want[0], "y")
        for k in g:
            same(g[k], want[1][k], k)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        both(off)
        end.record()
        torch.cuda.synchronize()
        took.append(begin.elapsed_time(end))
    assert took[0] <= 10 * took[1] + 10, took


@pytest.mark.parametrize("K,silu", [(4, True), (3, False)])
@pytest.mark.parametrize("dtype,batch,seqlen,dim,block", [
    (F32, 1, 16411, 1535, 32), (F32, 1, 26201, 1535, 64), (BF16, 1, 16411, 2560, 32), (BF16, 1, 26201, 2560, 64),
    (F32, 8, 1030, 2051, 32), (F32, 8, 2050, 2051, 64), (BF16, 8, 2047, 2050, 32), (BF16, 8, 4093, 2050, 64)])
def test_convolution_in_longer_blocks(ss, dtype, batch, seqlen, dim, block, K, silu):  # noqa: F811
    """Where at least 4096 waves have work, a wave has 32 or 64 tokens; dense, and packed requests that end
    around the borders of blocks, with states, infinities and NaN in the padding.  Channels are
    independent: some of every part of a row are compared.  A term of a parameter's gradient passes through
    its wave's tokens, 4 waves, a 16th of the workgroups along the tokens, 16 waves, and a rounding
    or two of its own."""
    r = np.random.default_rng(seqlen)
    off = None
    if batch == 1:
        around = [c for k in range(32, 400, 32) for c in (k - 3, k, k + 1)]
        off = np.array([0, 0, 0, *sorted({1, 2, 6, *around, *r.integers(400, seqlen - 41, 60)}), seqlen - 41, seqlen - 41], np.int32)
    seqs = batch if off is None else len(off) - 1
    x, dy = filled(batch * seqlen, dim, seed=1, dtype=dtype).view(batch, seqlen, dim), \
        filled(batch * seqlen, dim, seed=2, dtype=dtype).view(batch, seqlen, dim)
    w, b = normal(3, dim, K), normal(4, dim)
    h0, dlast = filled(seqs, dim, K - 1, seed=5, dtype=F32), filled(seqs, dim, K - 1, seed=6, dtype=F32)
    doff = None
    if off is not None:
        doff = torch.from_numpy(off).cuda()
        x[0, off[-1]:], dy[0, off[-1]:] = float("nan"), float("inf")
    y, last = ss.sscan_dwconv_fwd(x, w, b, silu=silu, initial_state=h0, offsets=doff, return_last_state=True)
    need = ss.dwconv_bwd_workspace_size(batch, seqlen, dim, K)
    room = torch.full((need + 4096,), 90, dtype=torch.uint8, device="cuda")
    g = ss.sscan_dwconv_bwd(x, w, dy, b, silu=silu, initial_state=h0, offsets=doff, dlast_state=dlast, workspace=room)
    assert bool((room[need:] == 90).all())
    cols = sorted({0, 1, 2, 3, 63, 64, 127, 128, 129, 255, 256, 257, dim // 2, *range(dim - 5, dim), *r.integers(0, dim, 16).tolist()})
    pick = lambda t: host(t[:, :, cols])
    args = (pick(x), host(w[cols]))
    kw = dict(silu=silu, initial_state=host(h0[:, cols]), offsets=off)
    want, wlast = layer.conv_fwd(*args, b=host(b[cols]), **kw)
    inside = np.array(args[0])
    if off is not None:
        inside[:, off[-1]:] = 0                     # (the bound is formed of all tokens)
    close(y[:, :, cols], want, layer.conv_fwd_error(inside, args[1], host(b[cols]), **kw), "y")
    np.testing.assert_array_equal(host(last[:, cols]), wlast)
    depth = block + 3 + -(-batch * -(-seqlen // (4 * block)) // 16) + 15 + 2
    ref = layer.conv_bwd(*args, pick(dy), b=host(b[cols]), dlast_state=host(dlast[:, cols]), depth=depth, **kw)
    close(g["dx"][:, :, cols], ref["dx"], ref["error"]["dx"], "dx")
    for k in ("dconv_w", "dconv_b"):
        close(g[k][cols], ref[k], ref["error"][k], k)
    close(g["dinitial_state"][:, cols], ref["dinitial_state"], ref["error"]["dinitial_state"], "dinitial_state")
    if off is not None:
        assert not bool(y[0, off[-1]:].any()) and not bool(g["dx"][0, off[-1]:].any())
    assert all(bool(t.isfinite().all()) for t in (y, last, *g.values()))
