"""The example block against a float64 restatement of it: outputs, every
gradient, training and the token-by-token pass.

The block chains about a dozen maps, each a sum of at most K = 256 products
(rounded with a relative error of 2^-24 a term, K 2^-24 of the largest in
all), and its normalisations multiply an error by up to about 4 (1 / the
spread of their input): 12 * 256 * 2^-24 * 4 = 7e-4 of the largest value of a
tensor bounds what fp32 can lose."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle

FP32_TOL = 7e-4


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "backbone_block.py")
    spec = importlib.util.spec_from_file_location("backbone_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(p, x, heads, groups, freqs, drop, seed, step):
    """The block in float64 torch operations; p and x float64 CPU tensors."""
    N, S, C = x.shape
    D = C // heads

    def norm(v, w, b, dims):
        mu = v.mean(dims, keepdim=True)
        var = (v - mu).square().mean(dims, keepdim=True)
        return (v - mu) / (var + 1e-5).sqrt() * w + b

    def keep(n, offset):
        m = torch.from_numpy(oracle.dropout_mask(n, drop, seed, offset))
        return m.double() * oracle.dropout_scale(drop)

    h = norm(x.view(N, S, groups, -1), 1.0, 0.0, (1, 3)).reshape(N, S, C)
    h = torch.nn.functional.silu(h * p["gn_w"] + p["gn_b"])
    qkv = (h @ p["wqkv"]).view(N, S, 3, heads, D)
    turns = torch.tensor([int(f) % 2 ** 64 / 2.0 ** 64 for f in freqs.tolist()],
                         dtype=torch.float64)
    ang = 2 * np.pi * torch.arange(S, dtype=torch.float64)[:, None] * turns
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]

    def rope(v, w):
        v = v / (v.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)

    q, k = rope(qkv[:, :, 0], p["q_norm"]), rope(qkv[:, :, 1], p["k_norm"])
    s = torch.einsum("nqhd,nkhd->nhqk", q, k) * D ** -0.5
    s = s.masked_fill(torch.ones(S, S, dtype=torch.bool).triu(1), float("-inf"))
    attn = torch.einsum("nhqk,nkhd->nqhd", s.softmax(-1), qkv[:, :, 2]).reshape(N, S, C)
    z = x + (attn @ p["wo"] + p["bo"]) * keep(N * S * C, 2 * step).view(N, S, C)
    y = norm(z, p["ln_w"], p["ln_b"], (2,))
    u = torch.nn.functional.silu(y @ p["w1"]) @ p["w2"]
    return z + (u + p["b2"]) * keep(N * S * C, 2 * step + 1).view(N, S, C)


def close(got, want, name):
    d = (got.detach().double().cpu() - want.detach()).abs().max().item()
    m = want.detach().abs().max().item()
    assert d <= FP32_TOL * m, (name, d, m)


@pytest.mark.gpu
def test_block_against_float64():
    m = load()
    block = m.Block(heads=2, head_dim=16, groups=4, hidden=48)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 9, 32, generator=g)
    dout = torch.randn(2, 9, 32, generator=g)
    xg = x.cuda().requires_grad_()
    out = block(xg, 0.25, 5, 3)
    got = torch.autograd.grad(out, [xg] + list(block.p.values()), dout.cuda())

    p64 = {k: v.detach().double().cpu().requires_grad_() for k, v in block.p.items()}
    x64 = x.double().requires_grad_()
    ref = plain(p64, x64, 2, 4, block.freqs.cpu(), 0.25, 5, 3)
    want = torch.autograd.grad(ref, [x64] + list(p64.values()), dout.double())
    close(out, ref, "out")
    for name, a, b in zip(["x"] + list(block.p), got, want):
        close(a, b, "d" + name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_trains_and_decodes(dtype):
    m = load()
    block = m.Block(dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(3, 21, 128, generator=g, device="cuda").to(dtype)
    losses = m.train(block, x, torch.tanh(x.roll(1, 1).float()).to(dtype), 12)
    assert losses[-1] < losses[0]
    with torch.no_grad():
        full = block(x).float()
    d = (full - block.decode(x).float()).abs().max().item()
    # the two passes differ in the order of their sums alone: in bf16 each of
    # the dozen maps may round its output the other way, by one step each
    tol = FP32_TOL if dtype == torch.float32 else 12 * 2 ** -7
    assert d <= tol * full.abs().max().item()
