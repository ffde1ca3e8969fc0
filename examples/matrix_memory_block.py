"""A pre-norm block with a matrix memory, trained and decoded with this library's operators.

    h = layer_norm(x);  P = h W^T + b  (q, k, v and gate slices of one projection)
    log decay = log sigmoid(mean of the head's gate slice + 4);  y = x + linear_attention(q, k, v, log decay)

Trains the block on a task that needs memory (each step's target is the mean of the sequence's earlier
inputs) for some steps of gradient descent, then decodes: the state of a prompt's end is carried token by
token, and must give what the whole sequence gives.

    python examples/matrix_memory_block.py            # needs an MI355X and the built library
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import recurrent_nets_amd as amd  # noqa: E402
from recurrent_nets_amd import slstm  # noqa: E402

GATE_BIAS = 4.0


class Block:
    """Parameters in float32 (the projection's weight is rounded to bfloat16 for its products)."""

    def __init__(self, width, heads, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.d = heads, width // heads
        self.norm_w, self.norm_b = torch.ones(width, device=device), torch.zeros(width, device=device)
        self.W = (torch.randn((4, width, width), generator=g) * width ** -0.5).to(device)
        self.b = torch.zeros((4, width), device=device)

    def project(self, x):
        """x (B, T, width) float32 -> the norm's statistics, h and the projection's four slices."""
        B, T, width = x.shape
        h, mean, rstd = amd.layer_norm_forward(x, self.norm_w, self.norm_b, out_dtype=torch.bfloat16, want_stats=True)
        P = amd.input_projection(h, self.W.bfloat16(), self.b)
        q, k, v, z = (P[:, :, i].view(B, T, self.heads, self.d) for i in range(4))
        z = z.mean(-1) + GATE_BIAS
        return (mean, rstd, h), q, k, v, z

    def forward(self, x, state=None):
        """(y, final state, what backward needs)."""
        stats, q, k, v, z = self.project(x)
        g = torch.nn.functional.logsigmoid(z)
        o, state1 = amd.linear_attention_forward(q, k, v, g, state, want_final_state=True)
        return x + o.view_as(x), state1, (x, stats, q, k, v, z, g, state)

    def backward(self, g_y, saved):
        """(dx, gradients of norm_w, norm_b, W, b)."""
        x, (mean, rstd, h), q, k, v, z, g, state = saved
        B, T, width = x.shape
        dP = torch.empty((B, T, 4, width), device=x.device)
        dq, dk, dv, dz = (dP[:, :, i].view(B, T, self.heads, self.d) for i in range(4))
        dg = amd.linear_attention_backward(q, k, v, g, g_y.view(B, T, self.heads, self.d), state, dq=dq, dk=dk, dv=dv)[3]
        dz.copy_((dg * torch.sigmoid(-z) / self.d)[..., None].expand_as(dz))
        dh, dW = slstm.input_projection_backward(h, self.W.bfloat16(), dP)
        dx, dw, db = amd.layer_norm_backward(x, dh, mean, rstd, self.norm_w)
        return g_y + dx, dw, db, dW, dP.sum((0, 1))

    def decode(self, x, state):
        """One token x (B, width) for each row; its state is updated in place."""
        _, q, k, v, z = self.project(x[:, None])
        g = torch.nn.functional.logsigmoid(z[:, 0]).contiguous()
        o = amd.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, state)
        return x + o.view_as(x)


def main(width=256, heads=4, batch=8, steps=96, iterations=60, lr=0.5, verbose=True):
    """Returns (first loss, last loss, largest difference of decoding from the whole sequence)."""
    block = Block(width, heads)
    gen = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for i in range(iterations):
        x = torch.randn((batch, steps, width), generator=gen, device="cuda")
        count = torch.arange(1, steps + 1, device="cuda")[:, None]
        target = x + x.cumsum(1) / count
        y, _, saved = block.forward(x)
        loss = ((y - target) ** 2).mean()
        _, dw, db, dW, dB = block.backward((y - target) * (2.0 / batch / steps), saved)
        for p, d in ((block.norm_w, dw), (block.norm_b, db), (block.W, dW), (block.b, dB)):
            p.sub_(d, alpha=lr / width)
        losses.append(float(loss))
        if verbose and i % 10 == 0:
            print(f"iteration {i}: loss {losses[-1]:.5f}", flush=True)

    x = torch.randn((batch, steps, width), generator=gen, device="cuda")
    whole, _, _ = block.forward(x)
    cut = steps // 3
    first, state, _ = block.forward(x[:, :cut].contiguous())
    tokens = [block.decode(x[:, t].contiguous(), state) for t in range(cut, steps)]
    far = float((torch.cat([first, torch.stack(tokens, 1)], 1) - whole).abs().max() / (whole - x).abs().max())
    if verbose:
        print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}; decoding is {far:.1e} off the whole sequence", flush=True)
    return losses[0], losses[-1], far


if __name__ == "__main__":
    main()
