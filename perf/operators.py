"""Cases of the backbone-block operators and their plain forms.

Four operators that a training program of a generative backbone chains:

* ``gn``       GroupNorm and an activation on channels-last tensors;
* ``dropout``  bias + dropout + add whose mask comes from a counter-based
               generator and is never stored;
* ``ln``       bias + dropout + add + LayerNorm with the same generator;
* ``rope``     RMSNorm of every query / key head followed by rotary positions,
               on the heads of a packed projection.

Each has a forward and a backward direction.  ``run`` computes them with
elementary torch operations, or, where ``own`` is true, through
``bwd_bn_pass_gb300.gbnorm``.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5

# Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
# as 1, 2, 3", 2011): multipliers and key increments.
M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
U32 = 0xFFFFFFFF


# --------------------------------------------------------------- the cases

def listed():
    return [
        # GroupNorm: the lowest-resolution level of a small U-Net at batch 1
        # (latency), the standard resolution of a latent backbone in both
        # directions, a whole batch in training (larger than L2), and an odd
        # channel count in fp32.
        {"name": "gn_fwd_small", "op": "gn", "dir": "fwd", "dtype": "f32",
         "N": 1, "H": 8, "W": 8, "C": 64, "G": 32, "act": "silu"},
        {"name": "gn_fwd", "op": "gn", "dir": "fwd", "dtype": "bf16",
         "N": 8, "H": 64, "W": 64, "C": 320, "G": 32, "act": "silu"},
        {"name": "gn_bwd_batch", "op": "gn", "dir": "bwd", "dtype": "bf16",
         "N": 64, "H": 64, "W": 64, "C": 512, "G": 32, "act": "silu"},
        {"name": "gn_bwd_ragged", "op": "gn", "dir": "bwd", "dtype": "f32",
         "N": 3, "H": 41, "W": 40, "C": 37, "G": 1, "act": "none"},
        # Dropout: the hidden tensor of a feed-forward layer on its way out,
        # and its gradient with the bias gradient; a short odd row.
        {"name": "dropout_fwd", "op": "dropout", "dir": "fwd", "dtype": "bf16",
         "R": 8192, "H": 8192, "p": 0.1, "bias": True, "residual": True},
        {"name": "dropout_bwd", "op": "dropout", "dir": "bwd", "dtype": "bf16",
         "R": 8192, "H": 1600, "p": 0.1, "bias": True, "residual": True},
        # LayerNorm: the repository's row workload in both directions, and an
        # odd width in fp32 (rows that are not whole 16-byte vectors).
        {"name": "ln_fwd", "op": "ln", "dir": "fwd", "dtype": "bf16",
         "R": 8192, "H": 1600, "p": 0.1},
        {"name": "ln_bwd", "op": "ln", "dir": "bwd", "dtype": "bf16",
         "R": 8192, "H": 1600, "p": 0.1},
        {"name": "ln_bwd_odd", "op": "ln", "dir": "bwd", "dtype": "f32",
         "R": 777, "H": 1001, "p": 0.25},
        # Rotary: one decoding step of 16 sequences far into a long context
        # (latency), a training batch, and its gradient.
        {"name": "rope_decode", "op": "rope", "dir": "fwd", "dtype": "bf16",
         "T": 16, "HQ": 32, "HK": 8, "D": 128, "rot": 128, "layout": "half",
         "norm": True, "far": True},
        {"name": "rope_fwd", "op": "rope", "dir": "fwd", "dtype": "bf16",
         "T": 16384, "HQ": 32, "HK": 8, "D": 128, "rot": 128, "layout": "half",
         "norm": True, "far": False},
        {"name": "rope_bwd_part", "op": "rope", "dir": "bwd", "dtype": "bf16",
         "T": 8192, "HQ": 16, "HK": 16, "D": 128, "rot": 64, "layout": "interleaved",
         "norm": True, "far": False},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _size(rng, lo, hi):
    """Log-spread; half the time a multiple of 8 where that fits."""
    v = _log(rng, lo, hi)
    if rng.random() < 0.5 and v >= 16:
        v -= v % 8
    return v


def draw(rng):
    op = rng.choice(["gn", "dropout", "ln", "rope"])
    case = {"op": op, "dir": rng.choice(["fwd", "bwd"]),
            "dtype": rng.choice(["bf16", "bf16", "f32"])}
    # no more bytes than the largest listed case of the operator
    limit = {"gn": 1 << 26, "dropout": 1 << 25, "ln": 1 << 24, "rope": 1 << 25}[op]
    if op == "gn":
        G = rng.choice([1, 4, 8, 16, 32, 32, 32, _log(rng, 1, 64)])
        Cg = _log(rng, 1, 48)
        H = _log(rng, 1, 128)
        W = _log(rng, 1, 128)
        N = _log(rng, 1, 64)
        while N * H * W * G * Cg > limit:
            N, H, W = max(1, N // 2), max(1, H - H // 4), max(1, W - W // 4)
        case.update(N=N, H=H, W=W, C=G * Cg, G=G, act=rng.choice(["silu", "silu", "none"]))
        if H * W * Cg < 2:
            case["H"] = 2
    elif op == "dropout":
        H = _size(rng, 1, 16384)
        R = _log(rng, 1, max(1, min(65536, limit // H)))
        case.update(R=R, H=H, p=rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.6), 3)]),
                    bias=rng.random() < 0.7, residual=rng.random() < 0.7)
    elif op == "ln":
        H = _size(rng, 8, 8192)
        R = _log(rng, 1, max(1, min(32768, limit // H)))
        case.update(R=R, H=H, p=rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.6), 3)]))
    else:
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256, 2 * _log(rng, 4, 128)])
        rot = rng.choice([D, D, D // 2 - (D // 2) % 2, 2 * rng.randint(1, D // 2)])
        HQ = _log(rng, 1, 64)
        HK = rng.choice([0, HQ, max(1, HQ // 4), 1])
        T = _log(rng, 1, max(1, min(32768, limit // (D * (HQ + HK)))))
        case.update(T=T, HQ=HQ, HK=HK, D=D, rot=max(2, rot),
                    layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.75,
                    far=rng.random() < 0.3)
        if case["dir"] == "bwd" and rng.random() < 0.7:
            case["norm"] = True
    return case


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _uniform(g, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(*shape, generator=g, device=DEV)


def _rng_of(seed):
    """Seed and offset of a training step's dropout stream."""
    r = np.random.default_rng(seed)
    return int(r.integers(0, 1 << 62)), int(r.integers(0, 1 << 40))


def inv_frequencies(rot, base=10000.0):
    """The rotary angle per position of every pair, in 64 bits."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    return base ** (-i / rot)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    op = case["op"]
    if op == "gn":
        N, S, C, G = case["N"], case["H"] * case["W"], case["C"], case["G"]
        # activations of a convolution: channels with offsets and spreads of
        # their own
        mu = _uniform(g, -2, 2, C)
        sd = _uniform(g, 0.25, 2, C)
        st["x"] = (mu + sd * _randn(g, N, case["H"], case["W"], C)).to(dt)
        st["gamma"] = _uniform(g, 0.5, 1.5, C)
        st["beta"] = 0.1 * _randn(g, C)
        if case["dir"] == "bwd":
            st["dy"] = _randn(g, N, case["H"], case["W"], C).to(dt)
            # the forward's saved statistics: mean (rounded and its remainder)
            # and 1/std of every sample and group
            stats = torch.empty(3, N, G, device=DEV)
            for n in range(N):
                xg = st["x"][n].double().view(S, G, C // G)
                m = xg.mean(dim=(0, 2))
                v = (xg - m.view(1, G, 1)).square().mean(dim=(0, 2))
                stats[0, n] = m.float()
                stats[1, n] = (1.0 / torch.sqrt(v + EPS)).float()
                stats[2, n] = (m - m.float().double()).float()
            st["stats"] = stats
    elif op in ("dropout", "ln"):
        R, H = case["R"], case["H"]
        st["seed"], st["offset"] = _rng_of(seed)
        has_bias = op == "ln" or case["bias"]
        has_res = op == "ln" or case["residual"]
        if op == "ln" or case["dir"] == "fwd":
            st["x"] = _randn(g, R, H).to(dt)
            st["bias"] = _randn(g, H).to(dt) if has_bias else None
            st["res"] = _randn(g, R, H).to(dt) if has_res else None
        if op == "ln":
            st["gamma"] = _uniform(g, 0.5, 1.5, H).to(dt)
            st["beta"] = (0.1 * _randn(g, H)).to(dt)
        if case["dir"] == "bwd":
            st["dy"] = _randn(g, R, H).to(dt)
            if op == "ln":
                z = _plain_dropout(st["x"], st["bias"], st["res"], case["p"], st["seed"],
                                   st["offset"]).double()
                m = z.mean(dim=1)
                st["mean"] = m.float()
                st["rstd"] = (1.0 / torch.sqrt((z - m[:, None]).square().mean(dim=1)
                                               + EPS)).float()
    else:
        T, HQ, HK, D = case["T"], case["HQ"], case["HK"], case["D"]
        # the packed projection: query, key and value heads of every token
        qkv = _randn(g, T, HQ + 2 * HK, D).to(dt)
        st["x"] = qkv[:, :HQ + HK]
        st["qkv"] = qkv
        hi = (1 << 20) if case["far"] else 4096
        if case["far"]:  # decoding: every sequence at a place of its own
            st["pos"] = torch.randint(0, hi, (T,), generator=g, device=DEV)
        else:            # training: whole sequences
            st["pos"] = torch.arange(T, device=DEV) % hi
        st["inv"] = inv_frequencies(case["rot"]).to(DEV)
        st["wq"] = _uniform(g, 0.5, 1.5, D).to(dt) if case["norm"] else None
        st["wk"] = _uniform(g, 0.5, 1.5, D).to(dt) if case["norm"] else None
        if case["dir"] == "bwd":
            st["dy"] = _randn(g, T, HQ + HK, D).to(dt)
            if case["norm"]:
                ms = st["x"].double().square().mean(dim=2)
                st["rstd"] = (1.0 / torch.sqrt(ms + EPS)).float()
        if own:
            from bwd_bn_pass_gb300 import gbnorm
            st["freqs"] = gbnorm.rope_frequencies(st["inv"])
    return st


# ------------------------------------------------------------ plain forms

def _keep16(p):
    """Of 2^16 equally likely 16-bit draws, how many keep the element."""
    return int(math.floor((1.0 - p) * 65536.0 + 0.5))


def _plain_keep(numel, p, seed, offset):
    """Whether each of numel elements is kept: element i takes the 16-bit
    piece i mod 8 (lowest first) of the four output words of block i // 8,
    whose counter is (block, offset) and whose key is the seed."""
    nb = (numel + 7) // 8
    b = torch.arange(nb, dtype=torch.int64, device=DEV)
    c = [b & U32, b >> 32, torch.full_like(b, offset & U32), torch.full_like(b, offset >> 32)]
    k0, k1 = seed & U32, seed >> 32
    for _ in range(10):
        p0, p1 = c[0] * M0, c[2] * M1
        c = [((p1 >> 32) & U32) ^ c[1] ^ k0, p1 & U32, ((p0 >> 32) & U32) ^ c[3] ^ k1, p0 & U32]
        k0, k1 = (k0 + W0) & U32, (k1 + W1) & U32
    pieces = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], dim=1)
    return (pieces < _keep16(p)).reshape(-1)[:numel]


def _scale(p):
    k = _keep16(p)
    return 65536.0 / k if k else 0.0


def _plain_dropout(x, bias, res, p, seed, offset):
    t = x.float()
    if bias is not None:
        t = t + bias.float()
    keep = _plain_keep(x.numel(), p, seed, offset).view(x.shape)
    t = torch.where(keep, t * _scale(p), torch.zeros_like(t))
    return t if res is None else res.float() + t


def _plain_gn(st, case):
    x, gamma, beta = st["x"], st["gamma"], st["beta"]
    N, S, C, G = case["N"], case["H"] * case["W"], case["C"], case["G"]
    xf = x.float().view(N, S, G, C // G)
    silu = case["act"] == "silu"
    if case["dir"] == "fwd":
        mean = xf.mean(dim=(1, 3), dtype=torch.float64)
        m0 = mean.float()
        m1 = (mean - m0.double()).float()
        xc = (xf - m0.view(N, 1, G, 1)) - m1.view(N, 1, G, 1)
        rstd = torch.rsqrt(xc.square().mean(dim=(1, 3), dtype=torch.float64) + EPS).float()
        pre = (xc * rstd.view(N, 1, G, 1)).view(N, S, C) * gamma + beta
        y = pre * torch.sigmoid(pre) if silu else pre
        return {"y": y.view(x.shape).to(x.dtype), "mean": m0, "rstd": rstd}
    m0, rstd, m1 = st["stats"]
    xh = ((xf - m0.view(N, 1, G, 1)) - m1.view(N, 1, G, 1)) * rstd.view(N, 1, G, 1)
    d = st["dy"].float().view(N, S, C)
    if silu:
        pre = xh.view(N, S, C) * gamma + beta
        s = torch.sigmoid(pre)
        d = d * (s * (1.0 + pre * (1.0 - s)))
    dgamma = (d * xh.view(N, S, C)).sum(dim=(0, 1), dtype=torch.float64).float()
    dbeta = d.sum(dim=(0, 1), dtype=torch.float64).float()
    gg = (d * gamma).view(N, S, G, C // G)
    a = gg.mean(dim=(1, 3), keepdim=True, dtype=torch.float64).float()
    b = (gg * xh).mean(dim=(1, 3), keepdim=True, dtype=torch.float64).float()
    dx = (gg - a - xh * b) * rstd.view(N, 1, G, 1)
    return {"dx": dx.reshape(x.shape).to(x.dtype), "dgamma": dgamma, "dbeta": dbeta}


def _plain_drop(st, case):
    if case["dir"] == "fwd":
        y = _plain_dropout(st["x"], st["bias"], st["res"], case["p"], st["seed"], st["offset"])
        return {"y": y.to(st["x"].dtype)}
    dy = st["dy"]
    keep = _plain_keep(dy.numel(), case["p"], st["seed"], st["offset"]).view(dy.shape)
    dx = torch.where(keep, dy.float() * _scale(case["p"]), torch.zeros(1, device=DEV))
    out = {"dx": dx.to(dy.dtype)}
    if case["bias"]:
        out["dbias"] = dx.sum(dim=0, dtype=torch.float64).to(dy.dtype)
    return out


def _plain_ln(st, case):
    x, dt = st["x"], st["x"].dtype
    z = _plain_dropout(x, st["bias"], st["res"], case["p"], st["seed"], st["offset"])
    if case["dir"] == "fwd":
        mean = z.mean(dim=1, keepdim=True)
        zc = z - mean
        rstd = torch.rsqrt(zc.square().mean(dim=1, keepdim=True) + EPS)
        y = zc * rstd * st["gamma"].float() + st["beta"].float()
        return {"y": y.to(dt), "z": z.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    rstd = st["rstd"][:, None]
    xh = (z - st["mean"][:, None]) * rstd
    dy = st["dy"].float()
    g = dy * st["gamma"].float()
    dz = rstd * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
    keep = _plain_keep(x.numel(), case["p"], st["seed"], st["offset"]).view(x.shape)
    dx = torch.where(keep, dz * _scale(case["p"]), torch.zeros_like(dz))
    cols = {"dgamma": dy * xh, "dbeta": dy, "dbias": dx}
    out = {"dx": dx.to(dt), "dresidual": dz.to(dt)}
    out.update({k: v.sum(dim=0, dtype=torch.float64).to(dt) for k, v in cols.items()})
    return out


def _rotate(v, cos, sin, rot, layout):
    """Rotary positions on the first rot of the last dimension; cos and sin
    are [T, 1, rot / 2]."""
    a = v[..., :rot]
    if layout == "half":
        u, w = a[..., :rot // 2], a[..., rot // 2:]
        r = torch.cat([u * cos - w * sin, w * cos + u * sin], dim=-1)
    else:
        u, w = a[..., 0::2], a[..., 1::2]
        r = torch.stack([u * cos - w * sin, w * cos + u * sin], dim=-1).flatten(-2)
    return torch.cat([r, v[..., rot:]], dim=-1)


def _plain_rope(st, case):
    x, dt, HQ = st["x"], st["x"].dtype, case["HQ"]
    ang = st["pos"].double()[:, None] * st["inv"]
    cos = torch.cos(ang).float()[:, None]
    sin = torch.sin(ang).float()[:, None]
    rot, lay = case["rot"], case["layout"]
    xf = x.float()
    if case["norm"]:
        w = torch.cat([st["wq"].float().expand(HQ, -1), st["wk"].float().expand(case["HK"], -1)])
    if case["dir"] == "fwd":
        if not case["norm"]:
            return {"y": _rotate(xf, cos, sin, rot, lay).to(dt)}
        rstd = torch.rsqrt(xf.square().mean(dim=2) + EPS)
        y = _rotate(xf * rstd[..., None] * w, cos, sin, rot, lay)
        return {"y": y.to(dt), "rstd": rstd}
    g = _rotate(st["dy"].float(), cos, -sin, rot, lay)
    if not case["norm"]:
        return {"dx": g.to(dt)}
    rstd = st["rstd"][..., None]
    xh = xf * rstd
    t = g * xh
    out = {"dwq": t[:, :HQ].sum(dim=(0, 1), dtype=torch.float64).to(dt)}
    if case["HK"]:
        out["dwk"] = t[:, HQ:].sum(dim=(0, 1), dtype=torch.float64).to(dt)
    gw = g * w
    out["dx"] = (rstd * (gw - xh * (gw * xh).mean(dim=2, keepdim=True))).to(dt)
    return out


_PLAIN = {"gn": _plain_gn, "dropout": _plain_drop, "ln": _plain_ln, "rope": _plain_rope}


# ------------------------------------------------- the framework's operators

def _own(st, case):
    from bwd_bn_pass_gb300 import gbnorm as F
    op, fwd = case["op"], case["dir"] == "fwd"
    if op == "gn":
        if fwd:
            y, stats = F.gn_nhwc_forward_train(st["x"], case["G"], st["gamma"], st["beta"], EPS,
                                               act=case["act"])
            return {"y": y, "mean": stats[0], "rstd": stats[1]}
        dx, dgamma, dbeta = F.gn_nhwc_backward(st["x"], st["dy"], st["stats"], st["gamma"],
                                               st["beta"], act=case["act"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "dropout":
        rng = (st["seed"], st["offset"])
        if fwd:
            return {"y": F.dropout_forward(st["x"], case["p"], rng, bias=st["bias"],
                                           residual=st["res"])}
        dx, dbias = F.dropout_backward(st["dy"], case["p"], rng, want_dbias=case["bias"])
        return {"dx": dx, "dbias": dbias} if case["bias"] else {"dx": dx}
    if op == "ln":
        rng = (st["seed"], st["offset"])
        if fwd:
            return F.layernorm_dropout_forward(st["x"], st["res"], case["p"], rng, st["gamma"],
                                               st["beta"], EPS, bias=st["bias"])
        return F.layernorm_dropout_backward(st["dy"], st["x"], st["res"], st["mean"], st["rstd"],
                                            st["gamma"], case["p"], rng, bias=st["bias"])
    if fwd:
        y, rstd = F.norm_rope_forward(st["x"], st["pos"], st["freqs"], st["wq"], st["wk"],
                                      q_heads=case["HQ"], eps=EPS, layout=case["layout"])
        return {"y": y, "rstd": rstd} if case["norm"] else {"y": y}
    dx, dwq, dwk = F.norm_rope_backward(st["dy"], st["x"], st["pos"], st["freqs"],
                                        st.get("rstd"), st["wq"], st["wk"],
                                        q_heads=case["HQ"], layout=case["layout"])
    out = {"dwq": dwq} if case["norm"] else {}
    if case["norm"] and case["HK"]:
        out["dwk"] = dwk
    out["dx"] = dx
    return out


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return _PLAIN[case["op"]](state, case)


# ------------------------------------------------------------------- work

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    op, fwd = case["op"], case["dir"] == "fwd"
    if op == "gn":
        n = case["N"] * case["H"] * case["W"] * case["C"]
        st = 8 * case["N"] * case["G"]
        act = 6 if case["act"] == "silu" else 0
        if fwd:
            return {"bytes": 2 * n * es + 8 * case["C"] + st, "flops": (7 + act) * n}
        return {"bytes": 3 * n * es + 16 * case["C"] + st, "flops": (14 + 2 * act) * n}
    if op == "dropout":
        n, H = case["R"] * case["H"], case["H"]
        bias = H * es if case["bias"] else 0
        if fwd:
            return {"bytes": (3 if case["residual"] else 2) * n * es + bias, "flops": 3 * n}
        return {"bytes": 2 * n * es + bias, "flops": 2 * n}
    if op == "ln":
        n, H = case["R"] * case["H"], case["H"]
        if fwd:
            return {"bytes": 4 * n * es + 3 * H * es + 8 * case["R"], "flops": 10 * n}
        return {"bytes": 5 * n * es + 5 * H * es + 8 * case["R"], "flops": 18 * n}
    rows = case["T"] * (case["HQ"] + case["HK"])
    n = rows * case["D"]
    extra = 8 * case["T"] + 4 * case["rot"]
    if case["norm"]:
        extra += 4 * rows + 2 * case["D"] * es
    if fwd:
        return {"bytes": 2 * n * es + extra, "flops": 7 * n}
    if case["norm"]:
        return {"bytes": 3 * n * es + extra + 2 * case["D"] * es, "flops": 12 * n}
    return {"bytes": 2 * n * es + extra, "flops": 3 * n}


# --------------------------------------------------- the definitions, 64 bits

def _exact_keep(numel, p, seed, offset):
    """The keep mask again, on the host with 64-bit unsigned products."""
    nb = (numel + 7) // 8
    out = np.empty((nb, 8), dtype=np.uint16)
    key = np.uint64(U32)
    s32 = np.uint64(32)
    for lo in range(0, nb, 1 << 20):
        b = np.arange(lo, min(nb, lo + (1 << 20)), dtype=np.uint64)
        x0, x1 = b & key, b >> s32
        x2 = np.full_like(b, offset & U32)
        x3 = np.full_like(b, (offset >> 32) & U32)
        for r in range(10):
            ka = np.uint64(((seed & U32) + r * W0) & U32)
            kb = np.uint64((((seed >> 32) & U32) + r * W1) & U32)
            a = x0 * np.uint64(M0)
            c = x2 * np.uint64(M1)
            x0, x1, x2, x3 = (c >> s32) ^ x1 ^ ka, c & key, (a >> s32) ^ x3 ^ kb, a & key
        words = np.stack([x0, x1, x2, x3], axis=1).astype("<u4")
        out[lo:lo + len(b)] = words.view("<u2")
    keep = out.reshape(-1)[:numel] < _keep16(p) if _keep16(p) < 65536 else np.ones(numel, bool)
    return torch.from_numpy(np.ascontiguousarray(keep)).to(DEV)


def _exact_gn(st, case):
    N, S, C, G = case["N"], case["H"] * case["W"], case["C"], case["G"]
    Cg = C // G
    cnt = S * Cg
    member = torch.zeros(C, G, dtype=torch.float64, device=DEV)
    member[torch.arange(C), torch.arange(C) // Cg] = 1.0
    gamma, beta = st["gamma"].double(), st["beta"].double()
    fwd = case["dir"] == "fwd"
    big = torch.empty(N, S, C, dtype=torch.float64, device=DEV)
    mean = torch.empty(N, G, dtype=torch.float64, device=DEV)
    rstd = torch.empty_like(mean)
    dgamma = torch.zeros(C, dtype=torch.float64, device=DEV)
    dbeta = torch.zeros_like(dgamma)
    for n in range(N):
        x = st["x"][n].reshape(S, C).double()
        if fwd:
            mg = (x.sum(dim=0)[None] @ member)[0] / cnt
            d = x - (member @ mg)
            rg = ((d * d).sum(dim=0)[None] @ member)[0].div(cnt).add(EPS).pow(-0.5)
            mean[n], rstd[n] = mg, rg
        else:
            mg = st["stats"][0, n].double() + st["stats"][2, n].double()
            rg = st["stats"][1, n].double()
            d = x - (member @ mg)
        r = member @ rg
        u = d * r
        pre = u * gamma + beta
        sg = 1.0 / (1.0 + torch.exp(-pre))
        if fwd:
            big[n] = pre * sg if case["act"] == "silu" else pre
            continue
        e = st["dy"][n].reshape(S, C).double()
        if case["act"] == "silu":
            e = e * (sg + pre * sg * (1.0 - sg))
        sb, sgm = e.sum(dim=0), (e * u).sum(dim=0)
        dbeta += sb
        dgamma += sgm
        k0 = member @ ((gamma * sb)[None] @ member)[0] / cnt
        k1 = member @ ((gamma * sgm)[None] @ member)[0] / cnt
        big[n] = r * (gamma * e - k0 - k1 * u)
    big = big.view(st["x"].shape)
    if fwd:
        return {"y": big, "mean": mean, "rstd": rstd}
    return {"dx": big, "dgamma": dgamma, "dbeta": dbeta}


def _exact_drop(st, case):
    src = st["x"] if case["dir"] == "fwd" else st["dy"]
    m = _exact_keep(src.numel(), case["p"], st["seed"], st["offset"]).view(src.shape).double()
    m *= _scale(case["p"])
    if case["dir"] == "bwd":
        dx = m * src.double()
        return {"dx": dx, "dbias": dx.sum(dim=0)} if case["bias"] else {"dx": dx}
    t = src.double()
    if st["bias"] is not None:
        t = t + st["bias"].double()
    t = t * m
    return {"y": t if st["res"] is None else t + st["res"].double()}


def _exact_ln(st, case):
    m = _exact_keep(st["x"].numel(), case["p"], st["seed"], st["offset"])
    m = m.view(st["x"].shape).double() * _scale(case["p"])
    z = st["res"].double() + m * (st["x"].double() + st["bias"].double())
    gamma = st["gamma"].double()
    H = case["H"]
    if case["dir"] == "fwd":
        mu = z.sum(dim=1) / H
        c = z - mu[:, None]
        r = (torch.einsum("ij,ij->i", c, c) / H + EPS) ** -0.5
        return {"y": c * r[:, None] * gamma + st["beta"].double(), "z": z, "mean": mu, "rstd": r}
    mu, r = st["mean"].double(), st["rstd"].double()
    c = z - mu[:, None]
    dy = st["dy"].double()
    gr = dy * gamma
    a = gr.sum(dim=1) / H
    b = torch.einsum("ij,ij->i", gr, c) * r / H
    dz = r[:, None] * (gr - a[:, None] - c * (r * b)[:, None])
    dx = dz * m
    return {"dx": dx, "dresidual": dz, "dgamma": torch.einsum("ij,ij,i->j", dy, c, r),
            "dbeta": dy.sum(dim=0), "dbias": dx.sum(dim=0)}


def _exact_rope(st, case):
    """Pairs as complex numbers: rotation is a product with exp(i angle)."""
    T, HQ, HK, D, rot = case["T"], case["HQ"], case["HK"], case["D"], case["rot"]
    turn = torch.polar(torch.ones(T, rot // 2, dtype=torch.float64, device=DEV),
                       st["pos"].double()[:, None] * st["inv"])[:, None]
    if case["layout"] == "half":
        i0 = torch.arange(rot // 2, device=DEV)
        i1 = i0 + rot // 2
    else:
        i0 = 2 * torch.arange(rot // 2, device=DEV)
        i1 = i0 + 1
    x = st["x"].double()
    heads = torch.arange(HQ + HK, device=DEV) < HQ

    def rotated(v, by):
        c = torch.complex(v[..., i0].contiguous(), v[..., i1].contiguous()) * by
        o = v.clone()
        o[..., i0], o[..., i1] = c.real, c.imag
        return o

    if case["norm"]:
        w = torch.where(heads[:, None], st["wq"].double(), st["wk"].double())
    if case["dir"] == "fwd":
        if not case["norm"]:
            return {"y": rotated(x, turn)}
        r = (torch.einsum("thd,thd->th", x, x) / D + EPS) ** -0.5
        return {"y": rotated(x * w * r[..., None], turn), "rstd": r}
    g = rotated(st["dy"].double(), turn.conj())
    if not case["norm"]:
        return {"dx": g}
    r = st["rstd"].double()
    dw = torch.einsum("thd,thd,th->hd", g, x, r)
    out = {"dwq": dw[:HQ].sum(dim=0)}
    if HK:
        out["dwk"] = dw[HQ:].sum(dim=0)
    gw = g * w
    s = torch.einsum("thd,thd->th", gw, x) / D
    out["dx"] = r[..., None] * gw - x * (s * r ** 3)[..., None]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    f = {"gn": _exact_gn, "dropout": _exact_drop, "ln": _exact_ln, "rope": _exact_rope}
    return f[case["op"]](st, case)
