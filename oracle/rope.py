"""RMSNorm of attention heads followed by rotary positions (oracle).

Test infrastructure only; see ``oracle/__init__.py``.

u = x / sqrt(mean(x^2) + eps) * w per head row (no norm where w is None); then
pair i of the first ``rot`` elements, as the complex number p + i q, is
multiplied by scale * exp(i * position * f_i).  The angle is reduced with exact
integer arithmetic: f_i is given as whole 2**-64ths of a turn.
"""

from fractions import Fraction

import numpy as np


def _angles(positions, freqs):
    """Exact angle of every (position, pair), as float64 radians."""
    out = np.empty((len(positions), len(freqs)))
    for a, p in enumerate(positions):
        for b, f in enumerate(freqs):
            t = (int(p) * int(f)) % (1 << 64)
            out[a, b] = 2.0 * np.pi * float(Fraction(t, 1 << 64))
    return out


def _pairs(rot, layout):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def _turn(v, ang, layout, scale):
    rot = 2 * ang.shape[1]
    i, j = _pairs(rot, layout)
    z = (v[..., i] + 1j * v[..., j]) * (scale * np.exp(1j * ang))[:, None, :]
    out = v.copy()
    out[..., i], out[..., j] = z.real, z.imag
    return out


def _weights(wq, wk, H, hq, D):
    w = np.ones((H, D))
    w[:hq] = np.asarray(wq, dtype=np.float64)
    if hq < H:
        w[hq:] = np.asarray(wk, dtype=np.float64)
    return w


def norm_rope_forward(x, positions, freqs, wq=None, wk=None, q_heads=None, eps=1e-5,
                      layout="half", scale=1.0):
    """x [T, H, D].  Returns dict y and rstd [T, H] (None without wq)."""
    x = np.asarray(x, dtype=np.float64)
    T, H, D = x.shape
    hq = H if q_heads is None else q_heads
    rstd = None
    if wq is not None:
        rstd = 1.0 / np.sqrt((x * x).mean(axis=2) + eps)
        x = x * rstd[..., None] * _weights(wq, wk, H, hq, D)
    return {"y": _turn(x, _angles(positions, freqs), layout, scale), "rstd": rstd}


def norm_rope_backward(dy, x, positions, freqs, rstd=None, wq=None, wk=None, q_heads=None,
                       layout="half", scale=1.0):
    """Returns dict dx, dwq, dwk (None without weights).  The gradient of the
    norm is taken through rstd as a function of the row: drstd/dx_j =
    -rstd^3 x_j / D."""
    dy = np.asarray(dy, dtype=np.float64)
    T, H, D = dy.shape
    hq = H if q_heads is None else q_heads
    g = _turn(dy, -_angles(positions, freqs), layout, scale)
    if wq is None:
        return {"dx": g, "dwq": None, "dwk": None}
    x = np.asarray(x, dtype=np.float64)
    r = np.asarray(rstd, dtype=np.float64)[..., None]
    w = _weights(wq, wk, H, hq, D)
    dw = (g * x * r).sum(axis=0)
    drstd = (g * w * x).sum(axis=2, keepdims=True)
    dx = g * w * r - drstd * r ** 3 * x / D
    return {"dx": dx, "dwq": dw[:hq].sum(axis=0), "dwk": dw[hq:].sum(axis=0) if hq < H else None}
