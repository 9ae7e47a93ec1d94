"""Decayed linear attention and the per-head norm with rotation from their definitions, in fp64 on
the CPU (numpy), token by token: what the GPU tests compare with.

Tolerances.  A rounding to a type is off by at most u = eps / 2 of the value (bf16 2^-8, fp16 2^-11,
fp32 2^-24), on average over the mantissa about 0.42 u in the root mean square.
  states (ht, dh0, the pool): fp32 sums, for every input type: 1e-5, the fp32 bar of the suite.
  o, dq, dk, dv fp32: 1e-5 as well.
  fp16: every product and sum is fp32, the result is rounded once: u = 2^-11, plus the fp32 bar.
  bf16: on the tensor cores the scores and the entering state are rounded to bf16 and the result once
    more; a score's rounding scales the terms near the token, the state's those far from it, so the
    sum has about the error of one operand rounding, and with the result's 2^(1/2) 0.42 2^-8 = 2.3e-3
    in the norm; 5e-3, the suite's bar, is twice that.
"""
from __future__ import annotations

import numpy as np

TOL_STATE = 1e-5
TOL = {"f32": 1e-5, "f16": 2.0 ** -11 + 1e-5, "bf16": 5e-3}


def decay(g):
    with np.errstate(over="ignore"):
        return np.exp(np.asarray(g, dtype=np.float64))


def fwd(q, k, v, g, h0, cu, scale):
    """o [T, H, V], ht [N, H, K, V] (rows past cu[-1] stay NaN)."""
    T, H, K = q.shape
    V, N = v.shape[2], len(cu) - 1
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    gam = decay(g)[:, None, None]
    o = np.full((T, H, V), np.nan)
    ht = np.zeros((N, H, K, V))
    for n in range(N):
        S = np.zeros((H, K, V)) if h0 is None else h0[n].astype(np.float64)
        for t in range(int(cu[n]), int(cu[n + 1])):
            S = gam * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
        ht[n] = S
    return o, ht


def bwd(q, k, v, g, h0, d_o, dht, cu, scale):
    """dq, dk, dv (NaN past cu[-1]) and dh0."""
    T, H, K = q.shape
    V, N = v.shape[2], len(cu) - 1
    q, k, v, d_o = (x.astype(np.float64) for x in (q, k, v, d_o))
    gam = decay(g)[:, None, None]
    dq, dk, dv = np.full((T, H, K), np.nan), np.full((T, H, K), np.nan), np.full((T, H, V), np.nan)
    dh0 = np.zeros((N, H, K, V))
    for n in range(N):
        S = np.zeros((H, K, V)) if h0 is None else h0[n].astype(np.float64)
        a, b = int(cu[n]), int(cu[n + 1])
        for t in range(a, b):
            S = gam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hkv,hv->hk", S, d_o[t])
        E = np.zeros((H, K, V)) if dht is None else dht[n].astype(np.float64)    # gamma G_{t+1}
        for t in range(b - 1, a - 1, -1):
            G = E + scale * q[t][:, :, None] * d_o[t][:, None, :]
            dk[t] = np.einsum("hkv,hv->hk", G, v[t])
            dv[t] = np.einsum("hkv,hk->hv", G, k[t])
            E = gam * G
        dh0[n] = E
    return dq, dk, dv, dh0


def turn(z, cos, sin, R, pairing, back=False):
    """z [T, H, D]; cos, sin [T, R / 2] (fp64)."""
    if R == 0:
        return z
    y = z.copy()
    c, s = cos[:, None, :], (-sin if back else sin)[:, None, :]
    ia, ib = ((slice(0, R // 2), slice(R // 2, R)) if pairing == "half" else (slice(0, R, 2), slice(1, R, 2)))
    a, b = z[..., ia], z[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def inv_norm(x, norm, eps):
    ss = np.square(x).sum(-1, keepdims=True)
    if norm == "rms":
        return 1.0 / np.sqrt(ss / x.shape[-1] + eps)
    return 1.0 / np.sqrt(ss + eps) if norm == "l2" else np.ones_like(ss)


def norm_rope(x, w, cos, sin, R, norm, eps, pairing):
    x = x.astype(np.float64)
    return turn(x * inv_norm(x, norm, eps) * (1.0 if w is None else w.astype(np.float64)), cos, sin, R, pairing)


def norm_rope_bwd(x, w, dy, cos, sin, R, norm, eps, pairing):
    """dx and the weight's gradient."""
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    w = np.ones(x.shape[-1]) if w is None else w.astype(np.float64)
    r = inv_norm(x, norm, eps)
    dz = turn(dy, cos, sin, R, pairing, back=True)
    dw = (dz * x * r).sum((0, 1))
    u = dz * w
    if norm == "none":
        return u, dw
    size = x.shape[-1] if norm == "rms" else 1
    return r * (u - x * r * r * (u * x).sum(-1, keepdims=True) / size), dw
