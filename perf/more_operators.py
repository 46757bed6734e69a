"""Measured cases of the operators around a recurrence in a layer: the norm with the residual's
addition, projections in 8-bit integers, and the short causal convolution.

Norm, for each token:

    s = x + residual, rounded to the residual's type (what is kept, and what is normed)
    r = 1 / sqrt(mean(s^2) + EPS)          y = s r w
    in 8 bits: scale = max(max|y| / 127, 2^-126) in float32, code = the whole number nearest to
    y / scale, ties to even

Product of rows in 8 bits, a [m, k] and weights b [n, k]:

    out = a_scale[m] b_scale[n] sum_k a[m, k] b[n, k] + bias[n]

Convolution of one channel, K taps, over dense batches [batch, seqlen, dim] or over requests
packed along one token axis (offsets[s] .. offsets[s + 1] are the tokens of request s; a
request may be empty; tokens past the last offset are padding, whose outputs are zero):

    v_t = b + sum_k w_k xx_{t - (K - 1) + k}          y_t = v_t, or v_t sigmoid(v_t)

where xx is x with the K - 1 tokens of the request's state before it.

A case's "op": "norm" (forward), "norm8" (output in 8 bits), "norm_train" (forward and
backward), "matmul" (rows that are in 8 bits already), "linear" (rows quantised, then the
product), "proj" (norm in 8 bits, then the product), "conv", "conv_train" (forward and
backward), "conv_step" (one token for every row against a pool of states).
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # One request's next token through a layer's norm and input projection: launch latency.
        dict(name="proj_one", op="proj", dtype="bf16", residual="bf16", rows=1, dim=2560, out=5120, bias=False, padded=True),
        # The same for a full decode batch, the projection to x and gate of a wide layer.
        dict(name="proj_decode", op="proj", dtype="bf16", residual="bf16", rows=256, dim=2560, out=10240, bias=False,
             padded=True),
        # A layer's output projection over a server's prefill, ragged in tokens, from what the
        # recurrence gave, into a float32 stream.
        dict(name="linear_packed", op="linear", dtype="bf16", outtype="f32", rows=16411, dim=2560, out=1280, bias=True,
             padded=True),
        # The input projection at the training batch's size, its rows in 8 bits already.
        dict(name="matmul_batch", op="matmul", dtype="bf16", rows=32768, dim=2048, out=4096, bias=False, padded=True),
        # The norm before a prefill's projection, its output kept in 8 bits.
        dict(name="norm8_packed", op="norm8", dtype="bf16", residual="bf16", rows=16411, dim=2560),
        # The norm of a forward at the training batch, with a float32 residual stream.
        dict(name="norm_batch", op="norm", dtype="bf16", residual="f32", rows=32768, dim=2048),
        # A training step's norm, forward and backward.
        dict(name="norm_train_batch", op="norm_train", dtype="bf16", residual="f32", rows=32768, dim=2048),
        # The same for a small layer in float32 at odd sizes.
        dict(name="norm_train_odd_f32", op="norm_train", dtype="f32", residual="f32", rows=4094, dim=1535),
        # A full decode batch on a pool of request states, some rows of the batch unused; the new
        # states go to other slots, so that a drafted token can be taken back.
        dict(name="conv_step_batch", op="conv_step", dtype="bf16", batch=256, slots=600, dim=5120, taps=4, silu=True, bias=True),
        # A server's prefill of ragged requests, some empty, with carried states and a padded tail,
        # inputs cut from one projection's output.
        dict(name="conv_packed", op="conv", dtype="bf16", batch=1, seqlen=16411, dim=2560, nseq=37, taps=4, silu=True,
             bias=True, fused=True, state=True),
        # A training step of a layer's convolution at the training batch.
        dict(name="conv_train_batch", op="conv_train", dtype="bf16", batch=8, seqlen=4096, dim=2048, nseq=0, taps=4,
             silu=True, bias=True, fused=False, state=False),
        # The same for a small layer in float32 at odd sizes, without the activation, documents packed.
        dict(name="conv_train_odd_f32", op="conv_train", dtype="f32", batch=1, seqlen=4094, dim=1535, nseq=23, taps=4,
             silu=False, bias=True, fused=True, state=True),
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "norm_train", "matmul", "linear", "proj", "conv", "conv_train", "conv_step"])
    dtype = rng.choice(["bf16", "f32"])
    elements = 32768 * 2048                      # no more than the training batch
    if op == "conv_step":
        batch = _log_between(rng, 1, 256)
        return dict(op=op, dtype=dtype, batch=batch, slots=2 * batch + rng.randint(1, 50), dim=_log_between(rng, 16, 5120),
                    taps=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.5)
    if op in ("conv", "conv_train"):
        dim = _log_between(rng, 16, 5120)
        tokens = _log_between(rng, 1, min(131072, elements // dim))
        packed = rng.random() < 0.5
        batch = 1 if packed else min(rng.choice([1, 1, 2, 3, 8]), tokens)
        return dict(op=op, dtype=dtype, batch=batch, seqlen=tokens // batch, dim=dim, nseq=_log_between(rng, 1, 64) if packed else 0,
                    taps=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.5,
                    fused=rng.random() < 0.5, state=rng.random() < 0.5)
    dim = _log_between(rng, 16, 5120)
    rows = _log_between(rng, 1, min(131072, elements // dim))
    residual = rng.choice(["none", dtype, "f32"])
    if op in ("norm", "norm8", "norm_train"):
        if op == "norm8":                        # its values come back in bfloat16
            dtype, residual = "bf16", rng.choice(["none", "bf16", "f32"])
        return dict(op=op, dtype=dtype, residual=residual, rows=rows, dim=dim)
    most = (32768 * 2048 * 4096) // (rows * dim)
    out = _log_between(rng, 16, max(16, min(10240, most, elements * 2 // rows)))
    if rng.random() < 0.5:                       # whole 16-byte rows, as most models have them
        dim, out = (dim + 15) // 16 * 16, (out + 15) // 16 * 16
    case = dict(op=op, dtype=dtype, rows=rows, dim=dim, out=out, bias=rng.random() < 0.5, padded=rng.random() < 0.7)
    if op == "proj":                             # in bfloat16: a code next to a border may go either way
        case.update(dtype="bf16", residual=rng.choice(["none", "bf16", "f32"]))
    if op == "linear":
        case.update(outtype=rng.choice(["bf16", "f32"]))
    return case


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _codes(v, padded):
    """Rows of v in 8 bits: codes (rows spaced by whole 16 bytes if padded) and scales."""
    scale = (v.abs().amax(1) / 127.0).clamp(min=2.0 ** -126)
    code = torch.round(v / scale[:, None]).to(torch.int8)
    if padded:
        room = torch.empty(v.shape[0], (v.shape[1] + 15) // 16 * 16, dtype=torch.int8, device="cuda")
        room[:, :v.shape[1]] = code
        code = room[:, :v.shape[1]]
    return code, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype, D = case["op"], _type(case["dtype"]), case["dim"]
    s = dict(op=op, dtype=dtype)
    # activations: unit normal with channels of larger and smaller size among them
    size = torch.exp(0.5 * _normal(gen, D))
    if op in ("norm", "norm8", "norm_train", "proj", "linear", "matmul"):
        M = case["rows"]
        x = _normal(gen, M, D) * size
        if op == "matmul":
            s["a"], s["a_scale"] = _codes(x, case["padded"])
            s["outtype"] = dtype
        else:
            s["x"] = x.to(dtype)
        if op not in ("linear", "matmul"):
            s["weight"] = 1.0 + 0.2 * _normal(gen, D)
            s["residual"] = None if case["residual"] == "none" else (2.0 * _normal(gen, M, D)).to(_type(case["residual"]))
            s["outtype"] = torch.bfloat16 if op == "proj" else dtype
        if op == "linear":
            s["outtype"] = _type(case["outtype"])
        if op in ("proj", "linear", "matmul"):
            N = case["out"]
            s["b"], s["b_scale"] = _codes(_normal(gen, N, D) * (D ** -0.5), case["padded"])
            s["bias"] = 0.1 * _normal(gen, N) if case["bias"] else None
        if op == "norm_train":
            s["dy"] = _normal(gen, M, D).to(dtype)
            s["dresidual"] = None if s["residual"] is None else _normal(gen, M, D).to(s["residual"].dtype)
        return s
    B, K = case["batch"], case["taps"]
    s.update(silu=case["silu"], w=_normal(gen, D, K) * (K ** -0.5), b=0.2 * _normal(gen, D) if case["bias"] else None)
    if op == "conv_step":
        s["x"] = (_normal(gen, B, D) * size).to(dtype)
        s["state"] = _normal(gen, case["slots"], D, K - 1) * size[:, None]
        # each request's slots before and after the token; the pool's last slot stays idle
        order = torch.randperm(case["slots"] - 1, generator=gen, device="cuda").to(torch.int32)
        s["slots"], s["slots_out"] = order[:B].clone(), order[B:2 * B].clone()
        if B > 16:                                # rows of the batch that hold no request
            s["slots"][torch.rand(B, generator=gen, device="cuda") < 0.05] = -1
        return s
    L = case["seqlen"]
    whole = _normal(gen, B, L, (2 if case["fused"] else 1) * D)       # fused: columns of one projection's output
    whole[..., :D] *= size
    s.update(x=whole.to(dtype)[..., :D], fused=case["fused"], offsets=None, initial=None, dlast=None, want_state=case["state"])
    rows = B
    if case["nseq"]:
        rows = case["nseq"]
        # ragged lengths: log-normal shares of the tokens, some requests empty, a padded tail
        share = torch.exp(_normal(gen, rows)) * (torch.rand(rows, generator=gen, device="cuda") > 0.15)
        share = torch.cumsum(share, 0) / share.sum().clamp_min(1e-6)
        used = L - min(L // 50, 40)
        ends = torch.floor(share * used + 0.5).clamp(max=used).to(torch.int32)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])
    if case["state"]:
        s["initial"] = _normal(gen, rows, D, K - 1) * size[:, None]
    if op == "conv_train":
        s["dy"] = _normal(gen, B, L, D).to(dtype)
        if case["state"]:
            s["dlast"] = _normal(gen, rows, D, K - 1)
    return s


# ---------------------------------------------------------------------------------------
# The plain forms: elementary operations in float32.
# ---------------------------------------------------------------------------------------

def _plain_norm(s):
    """(s as it is kept, s in float32, r, y in float32)."""
    kept = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = kept.float()
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return kept, v, r, v * r * s["weight"]


def _plain_norm_bwd(s, v, r):
    g = s["dy"].float()
    n = v * r
    dweight = (g * n).sum(0)
    g = g * s["weight"]
    d = r * (g - n * (g * n).mean(1, keepdim=True))
    if s["residual"] is None:
        return {"dx": d.to(s["dtype"]), "dweight": dweight}
    d = d + s["dresidual"].float()
    return {"dx": d.to(s["dtype"]), "dresidual": d.to(s["residual"].dtype), "dweight": dweight}


def _plain_quant(v):
    """Codes in float32, and scales.  The quotients are formed in 64 bits: some of them lie on
    the border between two codes, and the scale is the float32 number nearest to its own."""
    v = v.double()
    scale = (v.abs().amax(1, keepdim=True) / 127.0).float().clamp(min=2.0 ** -126)
    return torch.round(v / scale.double()).float(), scale


def _plain_product(s, a, a_scale):
    out = (a @ s["b"].float().t()) * a_scale * s["b_scale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(s["outtype"])


def _places(s, B, L):
    """Each token's sequence [B, L], its place in it and the places that follow it, and a mask of
    padding [B, L, 1]."""
    t = torch.arange(L, device="cuda")
    if s["offsets"] is None:
        return torch.arange(B, device="cuda")[:, None].expand(B, L), t.expand(B, L), (L - 1 - t).expand(B, L), None
    off = s["offsets"].long()
    row = torch.searchsorted(off[1:].contiguous(), t, right=True)
    pad = row >= off.numel() - 1
    row = row.clamp(max=off.numel() - 2)
    return row[None], (t - off[row])[None], (off[row + 1] - 1 - t)[None], pad[None, :, None]


def _before(s, x, row, place, j):
    """The input j tokens before each token: of the sequence, or of the state before it."""
    if j == 0:
        return x
    shifted = torch.nn.functional.pad(x, (0, 0, j, 0))[:, :x.shape[1]]
    K = s["w"].shape[1]
    if s["initial"] is None:
        start = torch.zeros(1, 1, 1, device="cuda")
    else:
        start = s["initial"][row, :, (K - 1 + place - j).clamp(0, K - 2)]
    return torch.where((place >= j)[..., None], shifted, start)


def _after(dv, left, j):
    """The gradient j tokens after each token, zero past its sequence's end."""
    shifted = torch.nn.functional.pad(dv, (0, 0, 0, j))[:, j:]
    return torch.where((left >= j)[..., None], shifted, torch.zeros_like(dv))


def _plain_conv(s):
    x = s["x"].float()
    B, L, D = x.shape
    K = s["w"].shape[1]
    row, place, left, pad = _places(s, B, L)
    if pad is not None:
        x = torch.where(pad, torch.zeros_like(x), x)
    taps = [_before(s, x, row, place, K - 1 - k) for k in range(K)]
    v = sum(taps[k] * s["w"][:, k] for k in range(K))
    if s["b"] is not None:
        v = v + s["b"]
    gate = torch.sigmoid(v)
    y = v * gate if s["silu"] else v
    if pad is not None:
        y = torch.where(pad, torch.zeros_like(y), y)
    out = {"y": y.to(s["dtype"])}
    off = s["offsets"]
    if off is None:
        starts = torch.arange(B, device="cuda") * L
        n = torch.full_like(starts, L)
    else:
        starts, n = off[:-1].long(), (off[1:] - off[:-1]).long()
    state_at = torch.arange(K - 1, device="cuda")             # places of the last state, from the sequence's start
    if s["want_state"]:
        place_of = n[:, None] - (K - 1) + state_at
        of_x = x.reshape(B * L, D)[(starts[:, None] + place_of).clamp(0, B * L - 1)].transpose(1, 2)
        of_initial = s["initial"].gather(2, (place_of + K - 1).clamp(0, K - 2)[:, None].expand(-1, D, -1))
        out["last_state"] = torch.where((place_of >= 0)[:, None], of_x, of_initial)
    if s["op"] == "conv":
        return out
    dv = s["dy"].float()
    if s["silu"]:
        dv = dv * (gate * (1.0 + v * (1.0 - gate)))
    if pad is not None:
        dv = torch.where(pad, torch.zeros_like(dv), dv)
    dx = sum(_after(dv, left, j) * s["w"][:, K - 1 - j] for j in range(K))
    if pad is not None:
        dx = torch.where(pad, torch.zeros_like(dx), dx)
    out["dw"] = torch.stack([(dv * tap).sum((0, 1)) for tap in taps], 1)
    if s["b"] is not None:
        out["db"] = dv.sum((0, 1))
    if s["dlast"] is not None:
        more = s["dlast"][row, :, (K - 2 - left).clamp(0, K - 2)]
        into = (left < K - 1)[..., None]
        dx = torch.where(into if pad is None else into & ~pad, dx + more, dx)
    out["dx"] = dx.to(s["dtype"])
    if s["initial"] is not None:
        flat = dv.reshape(B * L, D)

        def first(m):
            got = flat[(starts + m).clamp(max=B * L - 1)]
            return torch.where((n > m)[:, None], got, torch.zeros_like(got))

        din = torch.stack([sum(first(m) * s["w"][:, i - m] for m in range(i + 1)) for i in range(K - 1)], 2)
        over = state_at[None] - n[:, None]
        kept = s["dlast"].gather(2, over.clamp(min=0)[:, None].expand(-1, D, -1))
        out["dinitial"] = din + torch.where((over >= 0)[:, None], kept, torch.zeros_like(kept))
    return out


def _plain_conv_step(s):
    pool, idle = s["state"], s["state"].shape[0] - 1
    used = s["slots"] >= 0
    xx = torch.cat([pool[s["slots"].clamp(min=0).long()], s["x"].float()[..., None]], 2)
    v = (xx * s["w"]).sum(2)
    if s["b"] is not None:
        v = v + s["b"]
    y = v * torch.sigmoid(v) if s["silu"] else v
    # rows without a request write the idle last slot's own values to it
    pool[torch.where(used, s["slots_out"], torch.full_like(s["slots"], idle)).long()] = \
        torch.where(used[:, None, None], xx[..., 1:], pool[idle])
    return {"y": torch.where(used[:, None], y, torch.zeros_like(y)).to(s["dtype"]), "state": pool}


def _plain(s):
    op = s["op"]
    if op == "matmul":
        return {"out": _plain_product(s, s["a"].float(), s["a_scale"][:, None])}
    if op == "linear":
        return {"out": _plain_product(s, *_plain_quant(s["x"].float()))}
    if op == "conv_step":
        return _plain_conv_step(s)
    if op in ("conv", "conv_train"):
        return _plain_conv(s)
    kept, v, r, y = _plain_norm(s)
    out = {} if s["residual"] is None else {"residual": kept}
    if op == "proj":
        out["out"] = _plain_product(s, *_plain_quant(y))
    elif op == "norm8":
        code, scale = _plain_quant(y)
        out["y8"] = (code * scale).to(s["dtype"])
    else:
        out["y"] = y.to(s["dtype"])
        if op == "norm_train":
            out.update(_plain_norm_bwd(s, v, r))
    return out


# ---------------------------------------------------------------------------------------
# The framework's calls.
# ---------------------------------------------------------------------------------------

def _own(s):
    import selective_state_space_45_amd as ss
    op = s["op"]
    if op == "matmul":
        return {"out": ss.sscan_i8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], bias=s["bias"], dtype=s["outtype"])}
    if op == "linear":
        a, a_scale = ss.sscan_i8_quant(s["x"])
        return {"out": ss.sscan_i8_matmul(a, a_scale, s["b"], s["b_scale"], bias=s["bias"], dtype=s["outtype"])}
    if op == "conv_step":
        y = ss.sscan_dwconv_step(s["state"], s["x"], s["w"], conv_b=s["b"], silu=s["silu"], slots=s["slots"],
                                 slots_out=s["slots_out"])
        return {"y": y, "state": s["state"]}
    if op in ("conv", "conv_train"):
        y = ss.sscan_dwconv_fwd(s["x"], s["w"], conv_b=s["b"], silu=s["silu"], initial_state=s["initial"], offsets=s["offsets"],
                                return_last_state=s["want_state"])
        out = {"y": y}
        if s["want_state"]:
            out["y"], out["last_state"] = y
        if op == "conv":
            return out
        B, L, D = s["x"].shape
        into = None
        if s["fused"]:                            # its place in the gradient of the projection's output
            into = dict(dx=torch.empty(B, L, 2 * D, dtype=s["dtype"], device="cuda")[..., :D])
        g = ss.sscan_dwconv_bwd(s["x"], s["w"], s["dy"], conv_b=s["b"], silu=s["silu"], initial_state=s["initial"],
                                offsets=s["offsets"], dlast_state=s["dlast"], want_dbias=s["b"] is not None,
                                want_dinitial_state=s["initial"] is not None, out=into)
        out.update(dx=g["dx"], dw=g["dconv_w"])
        if s["b"] is not None:
            out["db"] = g["dconv_b"]
        if s["initial"] is not None:
            out["dinitial"] = g["dinitial_state"]
        return out
    eight = op in ("norm8", "proj")
    f = ss.sscan_rms_fwd(s["x"], s["weight"], residual=s["residual"], eps=EPS, want_y=not eight, want_codes=eight)
    out = {} if s["residual"] is None else {"residual": f["residual"]}
    if op == "proj":
        out["out"] = ss.sscan_i8_matmul(f["codes"], f["scales"], s["b"], s["b_scale"], bias=s["bias"], dtype=s["outtype"])
    elif op == "norm8":                           # the values that the codes stand for
        out["y8"] = torch.mul(f["codes"], f["scales"][:, None], out=torch.empty_like(s["x"]))
    else:
        out["y"] = f["y"]
        if op == "norm_train":
            kept = s["x"] if s["residual"] is None else f["residual"]
            g = ss.sscan_rms_bwd(kept, s["weight"], s["dy"], dresidual=s["dresidual"], eps=EPS,
                                 want_dresidual=s["residual"] is not None)
            out.update(dx=g["dx"], dweight=g["dweight"])
            if s["residual"] is not None:
                out["dresidual"] = g["dresidual"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e, op, D = (2 if case["dtype"] == "bf16" else 4), case["op"], case["dim"]
    if op in ("norm", "norm8", "norm_train", "proj", "linear", "matmul"):
        M = case["rows"]
        n = M * D
        kept = {"none": 0, "bf16": 2, "f32": 4}[case.get("residual", "none")]
        if op in ("proj", "linear", "matmul"):
            N = case["out"]
            to = 2 if op == "proj" else {"bf16": 2, "f32": 4}[case.get("outtype", case["dtype"])]
            rows = n * (1 if op == "matmul" else e + 2 * kept) + (4 * M if op == "matmul" else 0) + (4 * D if op == "proj" else 0)
            return {"bytes": rows + N * (D + (8 if case["bias"] else 4)) + M * N * to, "flops": 2 * M * N * D}
        moved = n * (2 * e + 2 * kept) + 4 * D
        if op == "norm_train":                    # dy and the gradient of what is kept read, the gradients written
            moved += n * (2 * e + 2 * kept) + 4 * D
        return {"bytes": moved, "flops": (18 if op == "norm_train" else 6) * n}
    K = case["taps"]
    params = 4 * D * (K + (1 if case["bias"] else 0))
    if op == "conv_step":
        n = case["batch"] * D
        return {"bytes": n * (2 * e + 8 * (K - 1)) + params + 8 * case["batch"], "flops": n * (2 * K + 6)}
    n = case["batch"] * case["seqlen"] * D
    rows = case["nseq"] or case["batch"]
    states = 8 * rows * D * (K - 1) if case["state"] else 0
    moved = 2 * e * n + params + states + (4 * (rows + 1) if case["nseq"] else 0)
    if op == "conv":
        return {"bytes": moved, "flops": n * (2 * K + 6)}
    return {"bytes": moved + 2 * e * n + params + states, "flops": n * (8 * K + 18)}


# ---------------------------------------------------------------------------------------
# The definition in 64 bits: each row or sequence by itself, gradients by differentiation.
# ---------------------------------------------------------------------------------------

def _exact_codes(y):
    """Codes and scales of 64-bit rows; the scale is a float32 number by definition."""
    scale = torch.maximum((y.abs().max(1).values / 127.0).float(), torch.tensor(2.0 ** -126, device="cuda")).double()
    return torch.round(y / scale[:, None]), scale


def _exact_rows(case, s):
    op = case["op"]
    if op == "matmul":
        codes, scale, out = s["a"].double(), s["a_scale"].double(), {}
    elif op == "linear":
        (codes, scale), out = _exact_codes(s["x"].double()), {}
    else:
        total = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        kept = total.to((s["x"] if s["residual"] is None else s["residual"]).dtype).double().requires_grad_()
        weight = s["weight"].double().requires_grad_()
        length = torch.sqrt(torch.linalg.vector_norm(kept, dim=1) ** 2 / kept.shape[1] + EPS)
        y = kept / length[:, None] * weight
        out = {} if s["residual"] is None else {"residual": total}
        if op == "norm":
            return {**out, "y": y.detach()}
        if op == "norm_train":
            loss = (y * s["dy"].double()).sum()
            if s["residual"] is not None:
                loss = loss + (kept * s["dresidual"].double()).sum()
            loss.backward()
            out.update(y=y.detach(), dx=kept.grad, dweight=weight.grad)
            if s["residual"] is not None:
                out["dresidual"] = kept.grad
            return out
        codes, scale = _exact_codes(y.detach())
        if op == "norm8":
            return {**out, "y8": codes * scale[:, None]}
    result = torch.matmul(codes, s["b"].double().t()) * torch.outer(scale, s["b_scale"].double())
    out["out"] = result if s["bias"] is None else result + s["bias"].double()
    return out


def _exact_act(v, silu):
    return v / (1.0 + torch.exp(-v)) if silu else v


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("conv"):
        return _exact_rows(case, s)
    K, D = case["taps"], case["dim"]
    w = s["w"].double().requires_grad_()
    b = (torch.zeros(D, dtype=torch.float64, device="cuda") if s["b"] is None else s["b"].double()).requires_grad_()
    if case["op"] == "conv_step":
        state, y = s["state"].double(), torch.zeros(case["batch"], D, dtype=torch.float64, device="cuda")
        new = state.clone()
        for n, (old, to) in enumerate(zip(s["slots"].tolist(), s["slots_out"].tolist())):
            if old >= 0:
                line = torch.cat([state[old], s["x"][n].double()[:, None]], 1)
                y[n] = _exact_act(b.detach() + torch.einsum("dk,dk->d", line, w.detach()), case["silu"])
                new[to] = line[:, 1:]
        return {"y": y, "state": new}
    x = s["x"].double().contiguous().requires_grad_()
    B, L, _ = x.shape
    rows = case["nseq"] or B
    h0 = (torch.zeros(rows, D, K - 1, dtype=torch.float64, device="cuda") if s["initial"] is None
          else s["initial"].double()).requires_grad_()
    off = None if s["offsets"] is None else s["offsets"].tolist()
    parts, lasts = [], []
    for n in range(rows):
        own_x = x[n] if off is None else x[0, off[n]:off[n + 1]]
        line = torch.cat([h0[n].t(), own_x])                          # the state's tokens, then the sequence
        size = own_x.shape[0]
        v = b + sum(line[k:k + size] * w[:, k] for k in range(K))
        parts.append(_exact_act(v, case["silu"]))
        lasts.append(line[size:].t())
    if off is None:
        y = torch.stack(parts)
    else:
        parts.append(torch.zeros(L - off[-1], D, dtype=torch.float64, device="cuda"))
        y = torch.cat(parts)[None]
    last = torch.stack(lasts)
    out = {"y": y.detach()}
    if case["state"]:
        out["last_state"] = last.detach()
    if case["op"] == "conv":
        return out
    loss = (y * s["dy"].double()).sum()
    if s["dlast"] is not None:
        loss = loss + (last * s["dlast"].double()).sum()
    loss.backward()
    out.update(dx=x.grad, dw=w.grad)
    if s["b"] is not None:
        out["db"] = b.grad
    if s["initial"] is not None:
        out["dinitial"] = h0.grad
    return out
