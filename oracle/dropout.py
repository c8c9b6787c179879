"""Dropout from a counter-based generator (oracle).

Test infrastructure only; see ``oracle/__init__.py``.

Generator: Philox4x32-10 as published (Salmon, Moraes, Dror, Shaw, "Parallel
random numbers: as easy as 1, 2, 3", 2011): ten rounds of two 32x32 -> 64-bit
products whose halves are xored with the other words and the key, which grows
by two Weyl constants a round.  Written here with Python integers.

Mask: element i takes the 16-bit piece i mod 8 of block i // 8, low half of a
word first; it is kept iff the piece is below floor((1 - p)*2**16 + 1/2).
"""

import numpy as np

_MASK = 0xFFFFFFFF


def philox4x32_10(counter, key):
    """One block: counter four and key two 32-bit words; four words out."""
    x0, x1, x2, x3 = counter
    k0, k1 = key
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = (b >> 32) ^ x1 ^ k0, b & _MASK, (a >> 32) ^ x3 ^ k1, a & _MASK
        k0, k1 = (k0 + 0x9E3779B9) & _MASK, (k1 + 0xBB67AE85) & _MASK
    return x0, x1, x2, x3


def dropout_threshold(p):
    return int(np.floor((1.0 - p) * 65536.0 + 0.5))


def dropout_scale(p):
    t = dropout_threshold(p)
    return 65536.0 / t if t else 0.0


def dropout_mask(n, p, seed, offset, start=0):
    """Keep decisions (bool) of elements start .. start + n - 1."""
    thr = dropout_threshold(p)
    out = np.empty(n, dtype=bool)
    block, pieces = None, None
    for k in range(n):
        i = start + k
        if i // 8 != block:
            block = i // 8
            w = philox4x32_10((block & _MASK, block >> 32, offset & _MASK, (offset >> 32) & _MASK),
                              (seed & _MASK, (seed >> 32) & _MASK))
            pieces = [h for v in w for h in (v & 0xFFFF, v >> 16)]
        out[k] = pieces[i % 8] < thr
    return out


def dropout_forward(x, p, seed, offset, bias=None, residual=None):
    """residual + keep*s*(x + bias); a dropped element adds exactly 0."""
    x = np.asarray(x, dtype=np.float64)
    keep = dropout_mask(x.size, p, seed, offset).reshape(x.shape)
    t = x if bias is None else x + np.asarray(bias, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        y = np.where(keep, t * dropout_scale(p), 0.0)
    return y if residual is None else np.asarray(residual, dtype=np.float64) + y


def dropout_backward(dy, p, seed, offset):
    """Returns dict dx and dbias (the column sums of dx over the rows)."""
    dy = np.asarray(dy, dtype=np.float64)
    keep = dropout_mask(dy.size, p, seed, offset).reshape(dy.shape)
    with np.errstate(invalid="ignore"):
        dx = np.where(keep, dy * dropout_scale(p), 0.0)
    return {"dx": dx, "dbias": dx.reshape(-1, dy.shape[-1]).sum(axis=0)}
