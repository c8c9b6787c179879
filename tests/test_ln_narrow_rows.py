"""LayerNorm backward over many narrow rows: one warp a row, so that a block has
fourteen groups of them, more than eight stages of the ring's rows, and a last
stage of one row."""

import numpy as np
import pytest
import torch

import oracle
from . import tolerances as tol


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


CASES = [(4505, 232, torch.bfloat16), (9001, 256, torch.bfloat16), (6007, 64, torch.bfloat16),
         (4505, 128, torch.float32), (9001, 48, torch.float32)]


@pytest.mark.gpu
@pytest.mark.parametrize("R,H,dtype", CASES)
@pytest.mark.parametrize("mask", ["none", "bytes", "drawn"])
def test_narrow_rows(gbn, R, H, dtype, mask):
    x, r, dy = (_rand((R, H), dtype, s) for s in (1, 2, 3))
    b = _rand((H,), dtype, 4)
    g = (_rand((H,), torch.float32, 5).abs() + 0.5).to(dtype)
    f64 = [t.double().numpy() for t in (dy, x, r, b, g)]
    seed, offset, p = 11, 12, 0.25
    if mask == "none":
        m, s = None, 1.0
    elif mask == "drawn":
        m, s = oracle.dropout_mask(R * H, p, seed, offset).reshape(R, H), oracle.dropout_scale(p)
    else:
        m, s = np.random.default_rng(6).random((R, H)) < 0.75, 1 / 0.75
    z = oracle.dropout_add(f64[1], f64[2], f64[3], m, s)
    mu, rs = (torch.tensor(v, dtype=torch.float32) for v in oracle.layer_norm_saved_stats(z, 1e-5))
    dev = [t.cuda() for t in (dy, x, r, b, g)]
    if mask == "drawn":
        out = gbn.layernorm_dropout_backward(dev[0], dev[1], dev[2], mu.cuda(), rs.cuda(), dev[4], p,
                                             (seed, offset), bias=dev[3])
    else:
        mk = None if m is None else torch.from_numpy(m).cuda()
        out = gbn.layernorm_backward(dev[0], dev[1], mu.cuda(), rs.cuda(), dev[4], residual=dev[2],
                                     bias=dev[3], mask=mk, dropout_scale=s)
    ref = oracle.fused_bias_dropout_add_layer_norm_backward(
        f64[0], f64[1], f64[2], f64[3], m, s, mu.double().numpy(), rs.double().numpy(), f64[4])
    name = "bf16" if dtype == torch.bfloat16 else "f32"
    for k in ("dx", "dresidual", "dgamma", "dbeta", "dbias"):
        tol.check(out[k], ref[k], f"narrow {R}x{H} {mask} {k}", name)
    assert gbn.get_device_status() == 0
