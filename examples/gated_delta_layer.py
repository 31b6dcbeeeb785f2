"""A residual sequence-mixing layer built on layer norm, the head norm with rotation and
the gated delta rule: trained for a few steps, then served -- packed prompts first, single
tokens on the resident states after.

    python examples/gated_delta_layer.py [--dim 512 --heads 8 --key-heads 4 ...]

The served outputs are compared with those of the whole sequences in one call,
and both are printed with the loss of every training step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_44_amd as ssm  # noqa: E402


class GatedDeltaLayer(torch.nn.Module):
    """x + W_o norm(o), where o is the gated delta rule on one fused projection of norm(x):
    queries and keys normed to length 1 and rotated, values, and per value head and token
    a decay and a step size."""

    def __init__(self, dim, heads, key_heads, kdim, vdim, max_positions, device, dtype):
        super().__init__()
        self.heads, self.key_heads, self.kdim, self.vdim = heads, key_heads, kdim, vdim
        at = dict(device=device, dtype=torch.float32)
        rows = 2 * key_heads * kdim + heads * vdim + 2 * heads
        param = lambda t: torch.nn.Parameter(t)
        self.w_in = param(torch.randn(rows, dim, **at).to(dtype) * dim ** -0.5)
        self.w_out = param(torch.randn(dim, heads * vdim, **at).to(dtype) * (heads * vdim) ** -0.5)
        self.norm_w, self.norm_b = param(torch.ones(dim, **at)), param(torch.zeros(dim, **at))
        self.out_w, self.out_b = param(torch.ones(vdim, **at)), param(torch.zeros(vdim, **at))
        # log decay = -rate softplus(. + bias): windows from a few tokens to a few hundred
        self.rate = param(torch.exp2(-torch.linspace(0, 7, heads, **at)))
        self.decay_bias = param(torch.zeros(heads, **at))
        self.register_buffer("unit", torch.full((kdim,), kdim ** -0.5, **at))
        turn = 10000.0 ** (-torch.arange(0, kdim, 2, **at) / kdim)
        angle = torch.arange(max_positions, **at)[:, None] * turn
        self.register_buffer("cos", angle.cos())
        self.register_buffer("sin", angle.sin())

    def operands(self, x):
        """q and k (not normed), v, log_decay, beta of [..., dim]."""
        p = torch.nn.functional.linear(ssm.LayerNorm.apply(x, self.norm_w, self.norm_b, 1e-5), self.w_in)
        g, h, k, v = self.key_heads, self.heads, self.kdim, self.vdim
        q, k, v, a, b = p.split([g * k, g * k, h * v, h, h], -1)
        decay = -self.rate * torch.nn.functional.softplus(a.float() + self.decay_bias)
        return (q.unflatten(-1, (g, -1)), k.unflatten(-1, (g, -1)), v.unflatten(-1, (h, -1)), decay,
                torch.sigmoid(b))

    def mixed(self, x, o):
        o = ssm.LayerNorm.apply(o, self.out_w, self.out_b, 1e-5)
        return x + torch.nn.functional.linear(o.flatten(-2), self.w_out)

    def forward(self, x, positions=None, cu_seqlens=None, h0=None):
        """x [batch, seqlen, dim], or [tokens, dim] packed with cu_seqlens.
        Returns y and the final states."""
        q, k, v, decay, beta = self.operands(x)
        q, k = ssm.QkNormRotate.apply(q, k, self.cos, self.sin, positions, self.unit, self.unit,
                                      1e-6, False)
        o, h = ssm.GatedDelta.apply(q, k, v, decay, beta, h0, 1.0, cu_seqlens)
        return self.mixed(x, o), h

    @torch.no_grad()
    def step(self, x, positions, h, slots=None):
        """One token per sequence, x [batch, dim]; the states h are updated in
        place."""
        q, k, v, decay, beta = self.operands(x)
        q, k = ssm.qk_norm_rotate(q, k, self.cos, self.sin, positions, self.unit, self.unit)
        return self.mixed(x, ssm.gated_delta_step(h, q, k, v, decay, beta, slots=slots))


def train(layer, steps, batch, seqlen, lr=0.01):
    """A few steps of gradient descent on recalling the token before last.
    Returns the losses."""
    g = torch.Generator(device=layer.w_in.device).manual_seed(1)
    opt = torch.optim.Adam(layer.parameters(), lr=lr)
    dim, losses = layer.w_in.shape[1], []
    for _ in range(steps):
        x = torch.randn(batch, seqlen, dim, generator=g, device=layer.w_in.device)
        x = x.to(layer.w_in.dtype)
        y, _ = layer(x)
        loss = (y[:, 2:].float() - x[:, :-2].float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        with torch.no_grad():
            layer.rate.clamp_(min=0.0)
        losses.append(loss.item())
    return losses


@torch.no_grad()
def serve(layer, prompts, new):
    """Packed prompts of the given lengths, then ``new`` tokens each, their
    states in slots of a larger pool.  Returns the largest difference from the
    whole sequences in one call, and the outputs' largest value."""
    device, dtype = layer.w_in.device, layer.w_in.dtype
    g = torch.Generator(device=device).manual_seed(2)
    dim, n = layer.w_in.shape[1], len(prompts)
    seqs = [torch.randn(p + new, dim, generator=g, device=device).to(dtype) for p in prompts]

    def packed(parts):
        lens = [p.shape[0] for p in parts]
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(device)
        pos = torch.cat([torch.arange(m, device=device) for m in lens])
        return layer(torch.cat(parts), pos, cu)

    y, h = packed([s[:p] for s, p in zip(seqs, prompts)])
    served = [list(part) for part in y.split(prompts)]
    pool = torch.zeros((2 * n, *h.shape[1:]), dtype=torch.float32, device=device)
    slots = torch.randperm(2 * n, generator=g, device=device)[:n].to(torch.int32)
    pool[slots.long()] = h
    for i in range(new):
        x = torch.stack([s[p + i] for s, p in zip(seqs, prompts)])
        pos = torch.tensor([p + i for p in prompts], device=device)
        for rows, row in zip(served, layer.step(x, pos, pool, slots)):
            rows.append(row)
    whole, _ = packed(seqs)
    served = torch.cat([torch.stack(rows) for rows in served])
    return (served.float() - whole.float()).abs().max().item(), whole.float().abs().max().item()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dim", type=int, default=512)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--key-heads", type=int, default=4)
    ap.add_argument("--kdim", type=int, default=64)
    ap.add_argument("--vdim", type=int, default=128)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--seqlen", type=int, default=256)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = GatedDeltaLayer(a.dim, a.heads, a.key_heads, a.kdim, a.vdim, 4096, "cuda:0",
                            torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    for i, loss in enumerate(train(layer, a.steps, a.batch, a.seqlen)):
        print(f"step {i}: loss {loss:.4f}")
    worst, size = serve(layer, [a.seqlen, 1, a.seqlen // 3 + 1], 8)
    print(f"served against whole sequences: largest difference {worst:.2e} (values up to {size:.2f})")


if __name__ == "__main__":
    main()
