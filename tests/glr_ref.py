"""The gated linear recurrence and the norms around a block from their definitions, in fp64 on the CPU (numpy), token by
token: what the GPU tests compare with.

Tolerances of the recurrence.  A result is rounded once to its type, off by at most u = eps / 2 of its value (bf16
2^-8, fp16 2^-11, fp32 2^-24; below fp16's least normal by 2^-25).  Before that, fp32: a decay, a mix and an input are off by some
units of 2^-24 (exp, reciprocal and root of a few ulp each, together at most 8), each step rounds once more, and
an error lives as long as the channel remembers, 1 / (1 - a) tokens: at most 10 2^-24 min(T, 1 / (1 - a)) of the largest
state.  A gradient multiplies two such sums and the derivatives of gate and mix: four times that.  drate adds up T of
its terms: its bound is of the sum of their magnitudes.
"""
from __future__ import annotations

import numpy as np

U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E32 = 2.0 ** -24


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def gates(r, rate, decay, mix):
    """log a, a, m, dm / dlog a."""
    if decay == "log":
        la = r
    elif decay == "sigmoid":
        la = -np.logaddexp(0, -r)
    else:
        la = -rate * sigmoid(r)
    with np.errstate(all="ignore"):
        a = np.exp(la)
        if mix == "one":
            return la, a, np.ones_like(a), np.zeros_like(a)
        if mix == "complement":
            return la, a, -np.expm1(la), -a
        m = np.sqrt(np.maximum(-np.expm1(2 * la), 0))
        return la, a, m, np.where(m > 0, -a * a / np.where(m > 0, m, 1), 0)


def fwd(x, r, i, rate, h0, cu, decay, mix):
    """h [T, D] and the state before each token (NaN past cu[-1]), ht [N, D]."""
    T, D = x.shape
    N = len(cu) - 1
    _, a, m, _ = gates(r, rate, decay, mix)
    u = x if i is None else x * sigmoid(i)
    h, prev = np.full((T, D), np.nan), np.full((T, D), np.nan)
    ht = np.zeros((N, D))
    with np.errstate(invalid="ignore", over="ignore"):
        for n in range(N):
            s = np.zeros(D) if h0 is None else h0[n].astype(np.float64)
            for t in range(cu[n], cu[n + 1]):
                prev[t] = s
                s = a[t] * s + m[t] * u[t]
                h[t] = s
            ht[n] = s
    return h, prev, ht


def bwd(x, r, i, rate, h0, d_o, dht, cu, decay, mix):
    """dx, dr, di, drate, dh0 and the sum of drate's terms' magnitudes."""
    T, D = x.shape
    N = len(cu) - 1
    la, a, m, dm = gates(r, rate, decay, mix)
    si = np.ones_like(x) if i is None else sigmoid(i)
    _, prev, _ = fwd(x, r, i, rate, h0, cu, decay, mix)
    G = np.full((T, D), np.nan)
    dh0 = np.zeros((N, D))
    for n in range(N):
        c = np.zeros(D) if dht is None else dht[n].astype(np.float64)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            G[t] = d_o[t] + c
            c = a[t] * G[t]
        dh0[n] = c
    dx = G * m * si
    di = G * m * x * si * (1 - si)
    dl = a * G * prev + G * x * si * dm
    terms = np.zeros_like(dl)
    if decay == "log":
        dr = dl
    elif decay == "sigmoid":
        dr = dl * sigmoid(-r)
    else:
        terms = -dl * sigmoid(r)
        dr = dl * la * sigmoid(-r)
    live = cu[-1]
    return dx, dr, di, terms[:live].sum(0), dh0, np.abs(terms[:live]).sum(0)


def memory(r, rate, decay, T):
    """Tokens that a channel remembers: 1 / (1 - a) of its mean decay, at most T."""
    _, a, _, _ = gates(r, rate, decay, "one")
    return float(min(T, 1.0 / max(1.0 - a.mean(0).max(), 1e-9)))


def check(name, got, ref, dtype, e32, scale=None):
    """Every value within its rounding and e32 of the largest."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, name
    if not ref.size:
        return
    top = np.abs(ref).max() if scale is None else scale
    bound = U[dtype] * np.abs(ref) * (1 + 2.0 ** -7) + e32 * top + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{name}: values that are not finite"
    worst = (err - bound).max()
    assert worst <= 0, f"{name}: off by {err.flat[(err - bound).argmax()]:.3e}, allowed {np.asarray(bound + 0 * err).flat[(err - bound).argmax()]:.3e}"


# ---------------------------------------------------------------- norms around a block
# Tolerances: each result is rounded once (U); before that fp32, some twenty roundings a value and sums of a row's D
# values, serial over at most 32 of them and a tree over the rest: 64 2^-24 of the largest value covers both.  The weights' gradients
# add up rows: as much of the sum of their terms' magnitudes.
E_NORM = 64 * E32


def philox(counter, key):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): counter [..., 4] and key [2] of 32-bit words."""
    c, k = [counter[..., j].astype(np.uint64) for j in range(4)], [np.uint64(key[0]), np.uint64(key[1])]
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> s32) ^ c[1] ^ k[0], q & low, (p >> s32) ^ c[3] ^ k[1], p & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(c, -1)


def keep(shape, p, seed, offset):
    """Dropout's factors: 0, or 65536 / (65536 - c) for kept values."""
    cut = int(np.floor(np.float64(np.float32(p)) * 65536 + 0.5))
    if cut == 0:
        return np.ones(shape)
    n = int(np.prod(shape))
    at = np.arange(-(-n // 8), dtype=np.uint64)
    seed, offset = np.uint64(seed % (1 << 64)), np.uint64(offset % (1 << 64))
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    ctr = np.stack([at & low, at >> s32, np.full_like(at, offset & low), np.full_like(at, offset >> s32)], -1)
    w = philox(ctr, (seed & low, seed >> s32))
    halves = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(-1)[:n]
    return (halves >= cut).reshape(shape) * (65536.0 / (65536 - cut))


def length(x, norm, eps):
    if norm in (None, "none"):
        return np.ones(x.shape[:-1] + (1,))
    s = (x * x).sum(-1, keepdims=True)
    return np.sqrt((s / x.shape[-1] if norm == "rms" else s) + eps)


def back(u, x, norm, eps):
    if norm in (None, "none"):
        return u
    l = length(x, norm, eps)
    n = x / l
    m = (u * n).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1)
    return (u - n * m) / l


def act(g, kind):
    """act(gate) and its derivative; 1 and 0 without gate."""
    if g is None:
        return 1.0, 0.0
    s = sigmoid(g)
    return {None: (g, np.ones_like(g)), "sigmoid": (s, s * (1 - s)), "silu": (g * s, s * (1 + g * (1 - s)))}[kind]


def block_fwd(y, gate, x, w_post, w_pre, f, post, pre, kind, eps):
    """xo, z; f: residual scale times dropout's factors."""
    w = 1.0 if w_post is None else w_post
    v = y / length(y, post, eps) * w * act(gate, kind)[0] * f
    xo = v if x is None else x + v
    return xo, xo / length(xo, pre, eps) * (1.0 if w_pre is None else w_pre)


def block_bwd(y, gate, x, dxo, dz, w_post, w_pre, f, post, pre, kind, eps):
    """dy, dgate, dx, dw_post, dw_pre and the sums of the weights' terms' magnitudes."""
    w1, w2 = (1.0 if w is None else w for w in (w_post, w_pre))
    a, da = act(gate, kind)
    n = y / length(y, post, eps)
    xo, _ = block_fwd(y, gate, x, w_post, w_pre, f, post, pre, kind, eps)
    d = np.zeros_like(xo) if dxo is None else dxo
    t2 = np.zeros_like(xo)
    if dz is not None:
        d = d + back(dz * w2, xo, pre, eps)
        t2 = dz * xo / length(xo, pre, eps)
    dn = d * f * a
    t1 = dn * n
    axes = tuple(range(xo.ndim - 1))
    return (back(dn * w1, y, post, eps), d * f * n * w1 * da, d, t1.sum(axes), t2.sum(axes), np.abs(t1).sum(axes).max(),
            np.abs(t2).sum(axes).max())
