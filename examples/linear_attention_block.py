"""A linear-attention block trained, then served, with the package's operators.

The block: x -> q, k, v; linear attention with a decay for each head; the norm
of each head's output with SiLU; the output projection. Training runs whole
sequences and their gradients; serving reads prompts of different lengths
packed back to back, which leaves a state for each sequence, and then feeds
one token of every sequence at a time to those states.

    python examples/linear_attention_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deltaproduct_householder_product_gb300 as dp  # noqa: E402


class Attend(torch.autograd.Function):
    """o [B,T,H,Dv] of whole sequences; the decay is a constant of the model."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay):
        o, _ = dp.linear_attention(q, k, v, log_decay, h_final=False)
        ctx.save_for_backward(q, k, v, log_decay)
        return o

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, log_decay = ctx.saved_tensors
        g = dp.linear_attention_backward(q, k, v, log_decay, d_o=d_o.contiguous(), want_dh0=False)
        return g["dq"], g["dk"], g["dv"], None


class HeadNorm(torch.autograd.Function):
    """silu(norm(x) weight + bias), x [rows, H D], statistics for each head."""

    @staticmethod
    def forward(ctx, x, weight, bias, heads):
        y, mean, rstd = dp.group_norm(x, weight, bias, groups=heads, act="silu")
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.heads = heads
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        g = dp.group_norm_backward(dy.contiguous(), x, weight, bias, mean, rstd, groups=ctx.heads, act="silu")
        return g["dx"], g["dweight"].to(weight.dtype), g["dbias"].to(bias.dtype), None


class Block(torch.nn.Module):
    def __init__(self, width, heads, head_dim, dtype=torch.bfloat16):
        super().__init__()
        self.heads, self.head_dim, inner = heads, head_dim, heads * head_dim
        self.qkv = torch.nn.Linear(width, 3 * inner, bias=False, dtype=dtype)
        self.weight = torch.nn.Parameter(torch.ones(inner, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(inner, dtype=dtype))
        self.out = torch.nn.Linear(inner, width, bias=False, dtype=dtype)
        # memories from 4 tokens to 512: log(1 - 2^-2) .. log(1 - 2^-9)
        self.register_buffer("log_decay", torch.log1p(-torch.exp2(-torch.linspace(2, 9, heads))))

    def project(self, x):
        """q, k, v [..., H, D]; q scaled as the readout wants it."""
        q, k, v = self.qkv(x).chunk(3, dim=-1)
        split = (*x.shape[:-1], self.heads, self.head_dim)
        return ((q * self.head_dim ** -0.5).reshape(split), k.reshape(split).contiguous(),
                v.reshape(split).contiguous())

    def finish(self, o, norm):
        y = norm(o.reshape(-1, self.heads * self.head_dim), self.weight, self.bias, self.heads)
        return self.out(y.view(*o.shape[:-2], -1))

    def forward(self, x, attend=Attend.apply, norm=HeadNorm.apply):
        """x [B,T,width], every sequence from an empty state."""
        return self.finish(attend(*self.project(x), self.log_decay), norm)

    @torch.no_grad()
    def prefill(self, x, lengths):
        """x [sum of lengths, width]: the outputs, and the states [N,H,D,D]."""
        cu = torch.tensor([0, *lengths], device=x.device).cumsum(0).int()
        o, states = dp.linear_attention_varlen(*self.project(x), self.log_decay, cu_seqlens=cu,
                                               max_seqlen=max(lengths))
        return self.finish(o, HeadNorm.apply), states

    @torch.no_grad()
    def step(self, x, states):
        """x [N,width], one token of each sequence; ``states`` move on in place."""
        return self.finish(dp.linear_attention_step(*self.project(x), self.log_decay, states), HeadNorm.apply)


def train(block, width, steps, batch, length, memory=0.75):
    """Learns a decaying average of the tokens so far (their first channel is a
    constant); returns the losses."""
    t = torch.arange(length, device="cuda")
    age = (t[:, None] - t[None, :]).float()
    average = torch.where(age >= 0, memory ** age.clamp(min=0), 0.0) * (1 - memory ** 2) ** 0.5
    opt = torch.optim.Adam(block.parameters(), lr=4e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn(batch, length, width, device="cuda", dtype=torch.bfloat16)
        x[..., 0] = 1
        loss = (block(x).float() - average @ x.float())[..., 1:].square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def serve(block, width, lengths, tokens):
    """Prompts, then ``tokens`` more of each; returns what the block answers for
    these, and for the same rows in whole sequences."""
    seqs = [torch.randn(n + tokens, width, device="cuda", dtype=torch.bfloat16) for n in lengths]
    _, states = block.prefill(torch.cat([s[:n] for s, n in zip(seqs, lengths)]), lengths)
    got = torch.stack([block.step(torch.stack([s[n + t] for s, n in zip(seqs, lengths)]), states)
                       for t in range(tokens)], dim=1)
    with torch.no_grad():
        whole = torch.stack([block(s[None])[0, n:] for s, n in zip(seqs, lengths)])
    return got, whole


def main(width=64, heads=4, head_dim=64, steps=200, batch=8, length=512, lengths=(700, 1, 0, 129), tokens=16):
    torch.manual_seed(0)
    block = Block(width, heads, head_dim).cuda()
    losses = train(block, width, steps, batch, length)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps of {batch} x {length} tokens")
    got, whole = serve(block, width, list(lengths), tokens)
    off = float((got.float() - whole.float()).square().mean().sqrt() / whole.float().square().mean().sqrt())
    print(f"{tokens} tokens each after prompts of {list(lengths)}: {off:.1e} from whole sequences (RMS)")
    return losses, off


if __name__ == "__main__":
    main()
