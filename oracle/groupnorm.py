"""GroupNorm with an activation on channels-last tensors (oracle).

Test infrastructure only; see ``oracle/__init__.py``.

Written out by the chain rule per sample and group over its S * C/G elements
(biased variance), pre = (x - mean)*rstd*gamma_c + beta_c, y = act(pre).
The backward differentiates through mean and variance explicitly.
"""

import numpy as np


def group_norm_act(pre, act, slope=0.01):
    if act in (None, "none"):
        return pre
    if act == "silu":
        return pre / (1.0 + np.exp(-pre))
    return np.where(pre > 0, pre, (0.0 if act == "relu" else slope) * pre)


def group_norm_act_gate(pre, act, slope=0.01):
    """d act / d pre."""
    if act in (None, "none"):
        return np.ones_like(pre)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-pre))
        return s + pre * s * (1.0 - s)
    return np.where(pre > 0, 1.0, 0.0 if act == "relu" else slope)


def _groups(x, G):
    x = np.asarray(x, dtype=np.float64)
    N, C = x.shape[0], x.shape[-1]
    return x.reshape(N, -1, G, C // G)


def _affine(v, C, fill):
    return np.full(C, fill) if v is None else np.asarray(v, dtype=np.float64)


def group_norm_forward(x, G, gamma=None, beta=None, eps=1e-5, act=None, slope=0.01):
    """x [N, ..., C].  Returns dict y, mean, rstd [N, G]."""
    x = np.asarray(x, dtype=np.float64)
    C = x.shape[-1]
    xg = _groups(x, G)
    mean = xg.mean(axis=(1, 3), keepdims=True)
    rstd = 1.0 / np.sqrt(((xg - mean) ** 2).mean(axis=(1, 3), keepdims=True) + eps)
    pre = ((xg - mean) * rstd).reshape(x.shape) * _affine(gamma, C, 1.0) + _affine(beta, C, 0.0)
    return {"y": group_norm_act(pre, act, slope), "mean": mean[:, 0, :, 0], "rstd": rstd[:, 0, :, 0],
            "pre": pre}


def group_norm_backward(x, dy, G, mean, rstd, gamma=None, beta=None, act=None, slope=0.01):
    """From the saved mean and rstd [N, G].  Returns dict dx, dgamma, dbeta."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    C = x.shape[-1]
    gm = _affine(gamma, C, 1.0)
    rho = np.asarray(rstd, dtype=np.float64)[:, None, :, None]
    cen = _groups(x, G) - np.asarray(mean, dtype=np.float64)[:, None, :, None]
    xhat = (cen * rho).reshape(x.shape)
    e = dy * group_norm_act_gate(xhat * gm + _affine(beta, C, 0.0), act, slope)
    axes = tuple(range(x.ndim - 1))
    g = _groups(e * gm, G)
    n = g.shape[1] * g.shape[3]
    dvar = (-0.5 * rho ** 3 * g * cen).sum(axis=(1, 3), keepdims=True)
    dmean = (-rho * g).sum(axis=(1, 3), keepdims=True)
    dx = g * rho + dvar * 2.0 * cen / n + dmean / n
    return {"dx": dx.reshape(x.shape), "dgamma": (e * xhat).sum(axis=axes),
            "dbeta": e.sum(axis=axes)}
