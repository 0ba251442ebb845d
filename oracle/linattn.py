"""fp64 CPU definitions of linear attention with a decay for each head and of
group norm with an activation, with their gradients: the recurrences as
written, token by token, in numpy. Run on the magnitudes of the inputs, the
same functions give the scales (sums of the magnitudes of all terms) that
errors are measured against.
"""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, np.float64) for x in xs]


def _lengths(lengths, B, L):
    return np.full(B, L) if lengths is None else np.clip(np.asarray(lengths, np.int64), 0, L)


def _decay(log_decay):
    return np.exp(np.asarray(log_decay, np.float64))  # exp(-inf) = 0: nothing is kept


def linattn(q, k, v, log_decay, scale=None, h0=None, lengths=None):
    """q [B, L, H, dk]; k, v [B, L, Hkv, dk / dv]. Returns y [B, L, H, dv], last_state [B, H, dk, dv]."""
    q, k, v, h0 = _f64(q, k, v, h0)
    B, L, H, dk = q.shape
    dv, per = v.shape[3], H // k.shape[2]
    scale = dk ** -0.5 if scale is None else scale
    lam = _decay(log_decay)[:, None, None]
    n = _lengths(lengths, B, L)
    y = np.zeros((B, L, H, dv))
    S = np.zeros((B, H, dk, dv)) if h0 is None else h0.copy()
    for b in range(B):
        for t in range(n[b]):
            kt, vt = np.repeat(k[b, t], per, 0), np.repeat(v[b, t], per, 0)
            S[b] = lam * S[b] + kt[:, :, None] * vt[:, None, :]
            y[b, t] = scale * np.einsum("hk,hkv->hv", q[b, t], S[b])
    return y, S


def linattn_step(state, q, k, v, log_decay, scale=None):
    y, S = linattn(q[:, None], k[:, None], v[:, None], log_decay, scale, state)
    return y[:, 0], S


def linattn_bwd(q, k, v, log_decay, dy, scale=None, h0=None, lengths=None, dlast=None):
    """Gradients by the recurrences of S (forwards), T = dS/dlog_decay and M (the gradient of S, backwards)."""
    q, k, v, dy, h0, dlast = _f64(q, k, v, dy, h0, dlast)
    B, L, H, dk = q.shape
    Hk, dv = k.shape[2], v.shape[3]
    per = H // Hk
    scale = dk ** -0.5 if scale is None else scale
    lam = _decay(log_decay)[:, None, None]
    n = _lengths(lengths, B, L)
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dlog_decay": np.zeros(H),
           "dh0": np.zeros((B, H, dk, dv))}
    for b in range(B):
        S = np.zeros((H, dk, dv)) if h0 is None else h0[b].copy()
        T = np.zeros_like(S)
        for t in range(n[b]):
            kt, vt = np.repeat(k[b, t], per, 0), np.repeat(v[b, t], per, 0)
            T = lam * (T + S)
            S = lam * S + kt[:, :, None] * vt[:, None, :]
            out["dq"][b, t] = scale * np.einsum("hkv,hv->hk", S, dy[b, t])
            out["dlog_decay"] += scale * np.einsum("hk,hkv,hv->h", q[b, t], T, dy[b, t])
        M = np.zeros_like(S) if dlast is None else dlast[b].copy()
        out["dlog_decay"] += (M * T).sum((1, 2))
        for t in range(n[b] - 1, -1, -1):
            kt, vt = np.repeat(k[b, t], per, 0), np.repeat(v[b, t], per, 0)
            M = M + scale * q[b, t][:, :, None] * dy[b, t][:, None, :]
            out["dk"][b, t] = np.einsum("hkv,hv->hk", M, vt).reshape(Hk, per, dk).sum(1)
            out["dv"][b, t] = np.einsum("hkv,hk->hv", M, kt).reshape(Hk, per, dv).sum(1)
            M = lam * M
        out["dh0"][b] = M
    return out


def _sig(x):
    return 1.0 / (1.0 + np.exp(-x))


def groupnorm(x, groups, weight=None, bias=None, z=None, act="none", eps=1e-5):
    """x [N, S, C] -> y, mean [N, G], rstd [N, G]."""
    x, weight, bias, z = _f64(x, weight, bias, z)
    N, S, C = x.shape
    xg = x.reshape(N, S, groups, C // groups)
    mean = xg.mean((1, 3))
    rstd = 1.0 / np.sqrt(((xg - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    xh = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    u = xh * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    y = u if act == "none" else u * _sig(u) if act == "silu" else u * z * _sig(z)
    return y, mean, rstd


def groupnorm_bwd(x, groups, weight=None, bias=None, z=None, act="none", dy=None, mean=None, rstd=None):
    x, weight, bias, z, dy, mean, rstd = _f64(x, weight, bias, z, dy, mean, rstd)
    N, S, C = x.shape
    D = C // groups
    w = np.ones(C) if weight is None else weight
    r = np.repeat(rstd, D, 1)[:, None]
    xh = (x - np.repeat(mean, D, 1)[:, None]) * r
    u = xh * w + (0.0 if bias is None else bias)
    out = {}
    if act == "silu":
        du = dy * _sig(u) * (1 + u * (1 - _sig(u)))
    elif act == "gate":
        du = dy * z * _sig(z)
        out["dz"] = dy * u * _sig(z) * (1 + z * (1 - _sig(z)))
    else:
        du = dy
    out["dweight"], out["dbias"] = (du * xh).sum((0, 1)), du.sum((0, 1))
    e = du * w

    def avg(a):
        return np.repeat(a.reshape(N, S, groups, D).mean((1, 3)), D, 1)[:, None]

    out["dx"] = r * (e - avg(e) - xh * avg(e * xh))
    return out
