"""One block of a generative backbone, trained and then run token by token.

    python examples/backbone_block.py [--dtype f32|bf16] [--steps 20]

The block's normalisation, positions and dropout are gbnorm calls, each with
its own backward; the projections and the attention are plain torch:

    h    = SiLU(GroupNorm(x))                     channels last
    q, k = rope(RMSNorm per head of h Wqkv)       on the packed projection
    z, y = LayerNorm of x + dropout(attn Wo + bo) mask drawn from a counter
    out  = z + dropout(SiLU(y W1) W2 + b2)        the same generator

The decoding pass sends one token of every sequence at a time through the
same calls (no rstd kept, a cache of rotated keys) and prints how far it is
from the full pass.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bwd_bn_pass_gb300 import gbnorm as G  # noqa: E402


class GroupNormSilu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, groups):
        y, stats = G.gn_nhwc_forward_train(x, groups, gamma, beta, act="silu")
        ctx.save_for_backward(x, stats, gamma, beta)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, stats, gamma, beta = ctx.saved_tensors
        dx, dgamma, dbeta = G.gn_nhwc_backward(x, dy.contiguous(), stats, gamma, beta, act="silu")
        return dx, dgamma, dbeta, None


class NormRope(torch.autograd.Function):
    """qkv [T, 3 * heads, D]: queries and keys normalised and turned, the
    values as they are; the gradient is one packed tensor again."""

    @staticmethod
    def forward(ctx, qkv, positions, freqs, wq, wk):
        heads = qkv.shape[1] // 3
        x = qkv[:, :2 * heads]
        qk, rstd = G.norm_rope_forward(x, positions, freqs, wq, wk, q_heads=heads)
        ctx.save_for_backward(x, positions, freqs, rstd, wq, wk)
        return qk, qkv[:, 2 * heads:].clone()

    @staticmethod
    def backward(ctx, dqk, dv):
        x, positions, freqs, rstd, wq, wk = ctx.saved_tensors
        T, H, D = x.shape
        dqkv = torch.empty(T, H + H // 2, D, dtype=x.dtype, device=x.device)
        _, dwq, dwk = G.norm_rope_backward(dqk.contiguous(), x, positions, freqs, rstd, wq, wk,
                                           q_heads=H // 2, dx=dqkv[:, :H])
        dqkv[:, H:] = dv
        return dqkv, None, None, dwq, dwk


class DropoutAddNorm(torch.autograd.Function):
    """(y, z) of z = residual + dropout(x + bias), y = LayerNorm(z); z carries
    on as the residual stream, so its gradient arrives besides y's."""

    @staticmethod
    def forward(ctx, x, residual, bias, gamma, beta, p, rng):
        o = G.layernorm_dropout_forward(x, residual, p, rng, gamma, beta, bias=bias)
        ctx.p, ctx.rng = p, rng
        ctx.save_for_backward(o["z"], o["mean"], o["rstd"], gamma)
        return o["y"], o["z"]

    @staticmethod
    def backward(ctx, dy, dz):
        z, mean, rstd, gamma = ctx.saved_tensors
        o = G.layernorm_dropout_backward(dy.contiguous(), z, None, mean, rstd, gamma, ctx.p,
                                         ctx.rng, saved_z=True, dz_extra=dz.float().contiguous())
        return o["dx"], o["dresidual"], o["dbias"], o["dgamma"], o["dbeta"], None, None


class DropoutAdd(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, bias, p, rng):
        ctx.p, ctx.rng = p, rng
        return G.dropout_forward(x, p, rng, bias=bias, residual=residual)

    @staticmethod
    def backward(ctx, dy):
        dy = dy.contiguous()
        dx, dbias = G.dropout_backward(dy, ctx.p, ctx.rng, want_dbias=True)
        return dx, dy, dbias, None, None


class Block:
    """heads * head_dim channels; parameters in ``self.p`` by name."""

    def __init__(self, heads=4, head_dim=32, groups=8, hidden=256, dtype=torch.float32, seed=0,
                 device="cuda"):
        C = heads * head_dim
        g = torch.Generator().manual_seed(seed)

        def make(*shape, scale=None, dt=dtype):
            t = torch.ones(shape) if scale is None else scale * torch.randn(shape, generator=g)
            return t.to(device=device, dtype=dt).requires_grad_()

        f32 = torch.float32
        self.heads, self.groups = heads, groups
        self.p = {
            "gn_w": make(C, dt=f32), "gn_b": make(C, scale=0.1, dt=f32),
            "wqkv": make(C, 3 * C, scale=C ** -0.5),
            "q_norm": make(head_dim), "k_norm": make(head_dim),
            "wo": make(C, C, scale=C ** -0.5), "bo": make(C, scale=0.1),
            "ln_w": make(C), "ln_b": make(C, scale=0.1),
            "w1": make(C, hidden, scale=C ** -0.5),
            "w2": make(hidden, C, scale=hidden ** -0.5), "b2": make(C, scale=0.1),
        }
        # a context four times the trained one, its slow pairs interpolated
        self.freqs = G.rope_frequencies(
            G.rope_inv_frequencies(head_dim, scaling="ramp", factor=4.0, original_length=256),
            device)

    def mix(self, q, k, v, causal):
        """Attention over [N, S, heads, D]."""
        q, k, v = (t.transpose(1, 2) for t in (q, k, v))
        s = (q @ k.transpose(-1, -2)).float() * q.shape[-1] ** -0.5
        if causal:
            s = s + torch.full(s.shape[-2:], float("-inf"), device=s.device).triu(1)
        return (torch.softmax(s, -1).to(v.dtype) @ v).transpose(1, 2).flatten(2)

    def tail(self, attn, x, drop, seed, step):
        """From the attention's output to the block's, rows [T, C].  The two
        dropouts of a step draw from offsets of their own."""
        p = self.p
        y, z = DropoutAddNorm.apply(attn @ p["wo"], x, p["bo"], p["ln_w"], p["ln_b"], drop,
                                    (seed, 2 * step))
        u = torch.nn.functional.silu(y @ p["w1"]) @ p["w2"]
        return DropoutAdd.apply(u, z, p["b2"], drop, (seed, 2 * step + 1))

    def __call__(self, x, drop=0.0, seed=0, step=0):
        """x [N, S, C], attention causal over S."""
        N, S, C = x.shape
        p = self.p
        h = GroupNormSilu.apply(x, p["gn_w"], p["gn_b"], self.groups)
        qkv = (h.view(N * S, C) @ p["wqkv"]).view(N * S, 3 * self.heads, -1)
        pos = torch.arange(S, device=x.device).repeat(N)
        qk, v = NormRope.apply(qkv, pos, self.freqs, p["q_norm"], p["k_norm"])
        q, k = (t.view(N, S, self.heads, -1) for t in qk.split(self.heads, 1))
        attn = self.mix(q, k, v.view(N, S, self.heads, -1), True)
        return self.tail(attn.view(N * S, C), x.view(N * S, C), drop, seed, step).view(N, S, C)

    @torch.no_grad()
    def decode(self, x):
        """The same map, one position of all sequences per step.  GroupNorm
        sees a whole sequence, so its output is made once, ahead."""
        N, S, C = x.shape
        p, heads = self.p, self.heads
        h, _ = G.gn_nhwc_forward_train(x, self.groups, p["gn_w"], p["gn_b"], act="silu")
        cache = torch.empty(2, N, S, heads, C // heads, dtype=x.dtype, device=x.device)
        pos = torch.empty(N, dtype=torch.int64, device=x.device)
        out = torch.empty_like(x)
        for s in range(S):
            qkv = (h[:, s] @ p["wqkv"]).view(N, 3 * heads, -1)
            pos.fill_(s)
            qk = qkv[:, :2 * heads]
            G.norm_rope_forward(qk, pos, self.freqs, p["q_norm"], p["k_norm"], q_heads=heads,
                                y=qk, want_rstd=False)
            cache[0, :, s], cache[1, :, s] = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
            attn = self.mix(qkv[:, None, :heads], cache[0, :, :s + 1], cache[1, :, :s + 1], False)
            out[:, s] = self.tail(attn[:, 0].contiguous(), x[:, s].contiguous(), 0.0, 0, 0)
        return out


def train(block, x, target, steps, drop=0.1, rate=0.02, seed=7):
    losses = []
    for step in range(steps):
        loss = (block(x, drop, seed, step).float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss, list(block.p.values()))
        with torch.no_grad():
            for w, g in zip(block.p.values(), grads):
                w -= rate * g
        losses.append(loss.item())
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="bf16")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--length", type=int, default=64)
    a = ap.parse_args()
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[a.dtype]
    block = Block(dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(8, a.length, 128, generator=g, device="cuda").to(dtype)
    target = torch.tanh(x.roll(1, 1).float()).to(dtype)
    losses = train(block, x, target, a.steps)
    print("loss", " ".join("%.4f" % v for v in losses))
    with torch.no_grad():
        full = block(x)
    worst = (full.float() - block.decode(x).float()).abs().max().item()
    print("token by token against the full pass: at most %.2g apart (largest value %.2g)"
          % (worst, full.float().abs().max().item()))


if __name__ == "__main__":
    main()
