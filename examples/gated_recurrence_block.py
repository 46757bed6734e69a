"""A small recurrent layer trained with its activations kept in 8 bits, then served.

The layer projects its tokens to x, the two gate pre-activations r and i and the output gate
z with one matrix product, runs the gated linear recurrence on the columns of that product,
and projects back.  Training packs documents of different lengths into one row, keeps a
state every 64 tokens and the activations in 8 bits, and returns the gradient of the whole
product as one tensor.  Serving prefills ragged requests in one call and decodes them
against a pool of states.

    python examples/gated_recurrence_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_45_amd as ss  # noqa: E402


class GatedRecurrence(torch.autograd.Function):
    """y of the recurrence on p = [x | r | i | z] ([1, tokens, 4 dim]), requests by offsets."""

    @staticmethod
    def forward(ctx, p, lam, r_bias, i_bias, offsets):
        x, r, i, z = p.split(p.shape[2] // 4, dim=2)
        shape = x.shape
        checkpoints = torch.empty(ss.glr_checkpoint_bytes(*shape) // 4, device=p.device)
        saved = torch.empty(ss.glr_saved_bytes(*shape, gated=True), dtype=torch.uint8, device=p.device)
        y = ss.sscan_glr_fwd(x, r, i, lam, r_bias=r_bias, i_bias=i_bias, z=z, offsets=offsets, checkpoints=checkpoints,
                             saved=saved)
        ctx.save_for_backward(lam, r_bias, i_bias, offsets, checkpoints, saved)   # and not p
        return y

    @staticmethod
    def backward(ctx, dy):
        lam, r_bias, i_bias, offsets, checkpoints, saved = ctx.saved_tensors
        dp = torch.empty(*dy.shape[:2], 4 * dy.shape[2], dtype=dy.dtype, device=dy.device)
        out = dict(zip(("dx", "dr", "di", "dz"), dp.split(dy.shape[2], dim=2)))
        g = ss.sscan_glr_bwd(lam, dy.contiguous(), checkpoints, saved=saved, gated=True, r_bias=r_bias, i_bias=i_bias,
                             offsets=offsets, want_dinitial_state=False, out=out)
        return dp, g["dlam"], g["dr_bias"], g["di_bias"], None


class Layer(torch.nn.Module):
    def __init__(self, width: int, dim: int):
        super().__init__()
        self.dim = dim
        self.inward = torch.nn.Linear(width, 4 * dim, bias=False, dtype=torch.bfloat16)
        self.outward = torch.nn.Linear(dim, width, bias=False, dtype=torch.bfloat16)
        # decays exp(-softplus(lam)) between 0.9 and 0.999
        a = torch.empty(dim).uniform_(0.9, 0.999)
        self.lam = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(a))))
        self.r_bias = torch.nn.Parameter(torch.zeros(dim))
        self.i_bias = torch.nn.Parameter(torch.zeros(dim))

    def forward(self, u, offsets):
        return self.outward(GatedRecurrence.apply(self.inward(u), self.lam, self.r_bias, self.i_bias, offsets))

    @torch.no_grad()
    def prefill(self, u, offsets):
        """Outputs of packed requests, and their states."""
        x, r, i, z = self.inward(u).split(self.dim, dim=2)
        y, state = ss.sscan_glr_fwd(x, r, i, self.lam, r_bias=self.r_bias, i_bias=self.i_bias, z=z, offsets=offsets,
                                    return_last_state=True)
        return self.outward(y), state

    @torch.no_grad()
    def decode(self, u, pool, slots):
        """One token for each row of a batch; slots[b] is row b's state in the pool, -1 for none."""
        x, r, i, z = self.inward(u).split(self.dim, dim=1)
        y = ss.sscan_glr_step(pool, x, r, i, self.lam, r_bias=self.r_bias, i_bias=self.i_bias, z=z, slots=slots)
        return self.outward(y)


def slow_average(u, offsets):
    """The task: out_t = 0.9 out_{t-1} + 0.1 u_t within each document, as a matrix product."""
    t = torch.arange(u.shape[1], device=u.device)
    doc = torch.searchsorted(offsets[1:].contiguous(), t.to(torch.int32), right=True)
    back = (t[:, None] - t[None, :]).clamp(min=0)
    weight = torch.where((t[:, None] >= t[None, :]) & (doc[:, None] == doc[None, :]), 0.1 * 0.9 ** back, 0.0)
    return weight @ u[0][None]


def main(steps: int = 60, width: int = 64, dim: int = 192, tokens: int = 1200, seed: int = 0, tell=print):
    """Returns the first and last losses and the largest difference of decoding from prefill."""
    torch.manual_seed(seed)
    layer = Layer(width, dim).cuda()
    opt = torch.optim.Adam(layer.parameters(), lr=2e-3)
    # documents of ragged lengths, some empty; the task: a slow average of the past tokens
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, tokens, (11,), generator=gen)).values
    offsets = torch.cat([torch.zeros(2, dtype=torch.int32), cuts.to(torch.int32), torch.tensor([tokens], dtype=torch.int32)])
    offsets = offsets.cuda()
    first = last = None
    for step in range(steps):
        u = torch.randn(1, tokens, width, device="cuda")
        target = slow_average(u, offsets)
        loss = (layer(u.bfloat16(), offsets).float() - target).square().mean() / target.square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        last = float(loss.detach())
        first = last if first is None else first
        if step % 10 == 0 or step == steps - 1:
            tell(f"step {step:3d}  loss {last:.4f}")
    # serve: prefill all but the last four tokens of three requests, decode the others
    n = [37, 130, 5]
    u = [torch.randn(k + 4, width, device="cuda").bfloat16() for k in n]
    whole = [layer.prefill(v[None], torch.tensor([0, v.shape[0]], dtype=torch.int32, device="cuda"))[0][0] for v in u]
    heads = torch.cat([v[:k] for v, k in zip(u, n)])[None]
    off = torch.tensor([0, 37, 167, 172], dtype=torch.int32, device="cuda")
    _, state = layer.prefill(heads, off)
    pool = torch.zeros(8, dim, device="cuda")
    slots = torch.tensor([6, 2, -1, 3], dtype=torch.int32, device="cuda")   # the third row of the batch is idle
    pool[[6, 2, 3]] = state
    worst = 0.0
    for t in range(4):
        row = torch.stack([u[0][n[0] + t], u[1][n[1] + t], torch.zeros_like(u[0][0]), u[2][n[2] + t]])
        y = layer.decode(row, pool, slots)
        for b, k in ((0, 0), (1, 1), (3, 2)):
            worst = max(worst, float((y[b].float() - whole[k][n[k] + t].float()).abs().max()))
    tell(f"decoding against one prefill: largest difference {worst:.4f}")
    return first, last, worst


if __name__ == "__main__":
    main()
