"""A small recurrent model trained with its activations kept in 8 bits, then served in 8 bits.

A layer adds the residual and takes its norm, projects its tokens to x, the two gate
pre-activations r and i and the output gate z with one matrix product, passes x through a short
causal convolution, runs the gated linear recurrence and projects back; a head follows a last
norm.  Training packs documents of different lengths into one row, keeps a state every 64 tokens
and the recurrence's inputs in 8 bits, and returns the gradient of the whole product as one
tensor.  Serving keeps the weights in 8 bits with a scale for each output, and the tokens with a
scale for each token: it prefills ragged requests in one call and decodes them against pools of
states.

    python examples/gated_recurrence_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_45_amd as ss  # noqa: E402


class Norm(torch.autograd.Function):
    """(norm of s, s), s = u + residual in float32."""

    @staticmethod
    def forward(ctx, u, residual, weight):
        out = ss.sscan_rms_fwd(u, weight, residual=residual, want_residual=True, residual_dtype=torch.float32)
        ctx.save_for_backward(out["residual"], weight)
        return out["y"], out["residual"]

    @staticmethod
    def backward(ctx, dy, ds):
        s, weight = ctx.saved_tensors
        g = ss.sscan_rms_bwd(s, weight, dy.contiguous(), dresidual=ds.contiguous(), want_dresidual=ctx.needs_input_grad[1])
        return g["dx"], g.get("dresidual"), g["dweight"]


class GatedRecurrence(torch.autograd.Function):
    """y of the convolution of x and the recurrence on p = [x | r | i | z] ([1, tokens, 4 dim]),
    requests by offsets."""

    @staticmethod
    def forward(ctx, p, conv_w, conv_b, lam, r_bias, i_bias, offsets):
        x, r, i, z = p.split(p.shape[2] // 4, dim=2)
        shape = x.shape
        checkpoints = torch.empty(ss.glr_checkpoint_bytes(*shape) // 4, device=p.device)
        saved = torch.empty(ss.glr_saved_bytes(*shape, gated=True), dtype=torch.uint8, device=p.device)
        xc = ss.sscan_dwconv_fwd(x, conv_w, conv_b, offsets=offsets)
        y = ss.sscan_glr_fwd(xc, r, i, lam, r_bias=r_bias, i_bias=i_bias, z=z, offsets=offsets, checkpoints=checkpoints,
                             saved=saved)
        ctx.save_for_backward(x.contiguous(), conv_w, conv_b, lam, r_bias, i_bias, offsets, checkpoints, saved)   # and not p
        return y

    @staticmethod
    def backward(ctx, dy):
        x, conv_w, conv_b, lam, r_bias, i_bias, offsets, checkpoints, saved = ctx.saved_tensors
        dp = torch.empty(*dy.shape[:2], 4 * dy.shape[2], dtype=dy.dtype, device=dy.device)
        dx, dr, di, dz = dp.split(dy.shape[2], dim=2)
        g = ss.sscan_glr_bwd(lam, dy.contiguous(), checkpoints, saved=saved, gated=True, r_bias=r_bias, i_bias=i_bias,
                             offsets=offsets, want_dinitial_state=False, out=dict(dr=dr, di=di, dz=dz))
        c = ss.sscan_dwconv_bwd(x, conv_w, g["dx"], conv_b, offsets=offsets, want_dinitial_state=False, out=dict(dx=dx))
        return dp, c["dconv_w"], c["dconv_b"], g["dlam"], g["dr_bias"], g["di_bias"], None


class Layer(torch.nn.Module):
    TAPS = 4

    def __init__(self, width: int, dim: int):
        super().__init__()
        self.dim = dim
        self.norm = torch.nn.Parameter(torch.ones(width))
        self.inward = torch.nn.Linear(width, 4 * dim, bias=False, dtype=torch.bfloat16)
        self.outward = torch.nn.Linear(dim, width, bias=False, dtype=torch.bfloat16)
        # the convolution starts near the identity
        self.conv_w = torch.nn.Parameter(0.1 * torch.randn(dim, self.TAPS) + torch.eye(self.TAPS)[-1])
        self.conv_b = torch.nn.Parameter(torch.zeros(dim))
        # decays exp(-softplus(lam)) between 0.9 and 0.999
        a = torch.empty(dim).uniform_(0.9, 0.999)
        self.lam = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(a))))
        self.r_bias = torch.nn.Parameter(torch.zeros(dim))
        self.i_bias = torch.nn.Parameter(torch.zeros(dim))

    def forward(self, u, residual, offsets):
        """(the layer's output, the residual stream before it)."""
        v, s = Norm.apply(u, residual, self.norm)
        y = GatedRecurrence.apply(self.inward(v), self.conv_w, self.conv_b, self.lam, self.r_bias, self.i_bias, offsets)
        return self.outward(y), s


class Model(torch.nn.Module):
    def __init__(self, width: int, dim: int, depth: int):
        super().__init__()
        self.layers = torch.nn.ModuleList(Layer(width, dim) for _ in range(depth))
        self.norm = torch.nn.Parameter(torch.ones(width))
        self.head = torch.nn.Linear(width, width, bias=False, dtype=torch.bfloat16)

    def forward(self, u, offsets):
        s = None
        for layer in self.layers:
            u, s = layer(u, s, offsets)
        return self.head(Norm.apply(u, s, self.norm)[0])


class Served:
    """The model with its weights in 8 bits, laid out once, and pools of `slots` states."""

    @torch.no_grad()
    def __init__(self, model: Model, slots: int):
        self.model = model
        self.weights = [[ss.sscan_i8_quant(m.weight) for m in (l.inward, l.outward)] for l in model.layers]
        self.head = ss.sscan_i8_quant(model.head.weight)
        dev = model.norm.device
        self.conv = [torch.zeros(slots, l.dim, l.TAPS - 1, device=dev) for l in model.layers]
        self.state = [torch.zeros(slots, l.dim, device=dev) for l in model.layers]

    def _run(self, u, mix):
        s = None
        for n, (layer, (inward, outward)) in enumerate(zip(self.model.layers, self.weights)):
            v = ss.sscan_rms_fwd(u, layer.norm, residual=s, want_y=False, want_codes=True, want_residual=True,
                                 residual_dtype=torch.float32)
            s = v["residual"]
            p = ss.sscan_i8_matmul(v["codes"], v["scales"], *inward)
            y = mix(n, layer, *p.split(layer.dim, dim=-1))
            u = ss.sscan_i8_matmul(*ss.sscan_i8_quant(y), *outward)
        v = ss.sscan_rms_fwd(u, self.model.norm, residual=s, want_y=False, want_codes=True, want_residual=False)
        return ss.sscan_i8_matmul(v["codes"], v["scales"], *self.head)

    @torch.no_grad()
    def prefill(self, u, offsets, slots):
        """Outputs of packed requests; request b's states go to slots[b] of the pools."""
        def mix(n, layer, x, r, i, z):
            x, conv = ss.sscan_dwconv_fwd(x, layer.conv_w, layer.conv_b, offsets=offsets, return_last_state=True)
            y, state = ss.sscan_glr_fwd(x, r, i, layer.lam, r_bias=layer.r_bias, i_bias=layer.i_bias, z=z, offsets=offsets,
                                        return_last_state=True)
            self.conv[n][slots], self.state[n][slots] = conv, state
            return y
        return self._run(u, mix)

    @torch.no_grad()
    def decode(self, u, slots):
        """One token for each row of a batch; slots[b] is row b's slot in the pools, -1 for none."""
        def mix(n, layer, x, r, i, z):
            x = ss.sscan_dwconv_step(self.conv[n], x, layer.conv_w, layer.conv_b, slots=slots)
            return ss.sscan_glr_step(self.state[n], x, r, i, layer.lam, r_bias=layer.r_bias, i_bias=layer.i_bias, z=z,
                                     slots=slots)
        return self._run(u, mix)


def slow_average(u, offsets):
    """The task: out_t = 0.9 out_{t-1} + 0.1 u_t within each document, as a matrix product."""
    t = torch.arange(u.shape[1], device=u.device)
    doc = torch.searchsorted(offsets[1:].contiguous(), t.to(torch.int32), right=True)
    back = (t[:, None] - t[None, :]).clamp(min=0)
    weight = torch.where((t[:, None] >= t[None, :]) & (doc[:, None] == doc[None, :]), 0.1 * 0.9 ** back, 0.0)
    return weight @ u[0][None]


def main(steps: int = 60, width: int = 64, dim: int = 192, tokens: int = 1200, seed: int = 0, tell=print, depth: int = 2):
    """Returns the first and last losses and the largest difference of decoding from prefill."""
    torch.manual_seed(seed)
    model = Model(width, dim, depth).cuda()
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    # documents of ragged lengths, some empty; the task: a slow average of the past tokens
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, tokens, (11,), generator=gen)).values
    offsets = torch.cat([torch.zeros(2, dtype=torch.int32), cuts.to(torch.int32), torch.tensor([tokens], dtype=torch.int32)])
    offsets = offsets.cuda()
    first = last = None
    for step in range(steps):
        u = torch.randn(1, tokens, width, device="cuda")
        target = slow_average(u, offsets)
        loss = (model(u.bfloat16(), offsets).float() - target).square().mean() / target.square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        last = float(loss.detach())
        first = last if first is None else first
        if step % 10 == 0 or step == steps - 1:
            tell(f"step {step:3d}  loss {last:.4f}")
    # serve: prefill all but the last four tokens of three requests, decode the others
    served = Served(model, slots=8)
    n = [37, 130, 5]
    u = [torch.randn(k + 4, width, device="cuda").bfloat16() for k in n]
    index = lambda *v, dtype=torch.int32: torch.tensor(v, dtype=dtype, device="cuda")
    whole = [served.prefill(v[None], index(0, v.shape[0]), index(0, dtype=torch.int64))[0] for v in u]
    served.prefill(torch.cat([v[:k] for v, k in zip(u, n)])[None], index(0, 37, 167, 172), index(6, 2, 3, dtype=torch.int64))
    slots = index(6, 2, -1, 3)      # the third row of the batch is idle
    worst = 0.0
    for t in range(4):
        row = torch.stack([u[0][n[0] + t], u[1][n[1] + t], torch.zeros_like(u[0][0]), u[2][n[2] + t]])
        y = served.decode(row, slots)
        for b, k in ((0, 0), (1, 1), (3, 2)):
            worst = max(worst, float((y[b].float() - whole[k][n[k] + t].float()).abs().max()))
    tell(f"decoding against one prefill: largest difference {worst:.4f}")
    return first, last, worst


if __name__ == "__main__":
    main()
