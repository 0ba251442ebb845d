"""fp64 CPU definitions of the gated linear recurrence, of the norms around a
block with the residual sum, and of rotary positions, with their gradients:
the formulas as written, token by token, in numpy.
"""
from __future__ import annotations

import numpy as np

from .linattn import _f64, _lengths


def sigmoid(v):
    t = np.exp(-np.abs(v))
    return np.where(v >= 0, 1, t) / (1 + t)


def silu(z):
    return z * sigmoid(z)


def silu_grad(z):
    return sigmoid(z) * (1 + z * sigmoid(-z))


def gated_terms(x, g, r=None, A=None):
    """a, 1 - a, w (the weight beside the gate) and b = w sigmoid(g) x (mix: u x) of every token."""
    x, g, r, A = _f64(x, g, r, A)
    v = sigmoid(g)
    if r is None:
        return sigmoid(-g), v, np.ones_like(v), v * x
    l = A * sigmoid(r)
    w = np.sqrt(-np.expm1(2 * l))
    return np.exp(l), -np.expm1(l), w, w * v * x


def _walk(a, b, h0, n):
    """h before and after each token of h = a h + b, frozen behind entry i's n[i] tokens."""
    B, L, D = a.shape
    h = np.zeros((B, D)) if h0 is None else np.array(h0, np.float64)
    before, after = np.empty((B, L, D)), np.empty((B, L, D))
    for t in range(L):
        before[:, t] = h
        h = np.where((t < n)[:, None], a[:, t] * h + b[:, t], h)
        after[:, t] = h
    return before, after, h


def gated(x, g, r=None, A=None, z=None, h0=None, lengths=None):
    """x, g, r, z [B, L, D]; A [D]. Returns y [B, L, D], last_state [B, D], the states before the tokens."""
    a, _, _, b = gated_terms(x, g, r, A)
    B, L, D = a.shape
    n = _lengths(lengths, B, L)
    before, after, last = _walk(a, b, h0, n)
    y = after if z is None else after * silu(np.asarray(z, np.float64))
    return np.where((np.arange(L) < n[:, None])[..., None], y, 0.0), last, before


def gated_bwd(x, g, dy, r=None, A=None, z=None, h0=None, lengths=None, dlast=None):
    """Gradients for sum(y dy) + sum(last_state dlast): dx, dg, dh0 and, where there are such inputs, dr, dA, dz."""
    a, _, w, b = gated_terms(x, g, r, A)
    x, g, dy, r, A, z, dlast = _f64(x, g, dy, r, A, z, dlast)
    B, L, D = a.shape
    n = _lengths(lengths, B, L)
    here = (np.arange(L) < n[:, None])[..., None]
    before, after, _ = _walk(a, b, h0, n)
    out = {}
    dy = np.where(here, dy, 0.0)
    d = dy
    if z is not None:
        out["dz"] = dy * after * silu_grad(z)
        d = dy * silu(z)
    G = np.zeros((B, L, D))
    C = np.zeros((B, D)) if dlast is None else dlast.copy()
    for t in range(L - 1, -1, -1):
        on = (t < n)[:, None]
        G[:, t] = np.where(on, d[:, t] + C, 0.0)
        C = np.where(on, a[:, t] * G[:, t], C)
    out["dh0"] = C
    v = sigmoid(g)
    out["dx"] = G * w * v
    if r is None:
        out["dg"] = G * (x - before) * v * sigmoid(-g)
        return out
    out["dg"] = G * w * x * v * sigmoid(-g)
    slope = np.divide(a * a, w, out=np.zeros_like(w), where=w > 0)
    dl = G * (a * before - slope * v * x)
    out["dr"] = dl * A * sigmoid(r) * sigmoid(-r)
    out["dA"] = (dl * sigmoid(r)).sum((0, 1))
    return out


def _norm(v, kind, weight, bias, eps):
    mean = v.mean(1) if kind == "layer" else np.zeros(len(v))
    rstd = 1 / np.sqrt(((v - mean[:, None]) ** 2).mean(1) + eps)
    return (v - mean[:, None]) * rstd[:, None] * weight + bias, mean, rstd


def _params(C, *ps):
    return [np.asarray(p, np.float64) if p is not None else np.full(C, d) for p, d in zip(ps, (1.0, 0.0, 1.0, 0.0))]


def _gate_rows(gate, R, C):
    return np.ones((R, C)) if gate is None else np.repeat(np.asarray(gate, np.float64), R // len(gate), 0)


def addnorm(x, res=None, pre="rms", pre_weight=None, pre_bias=None, post="none", post_weight=None, post_bias=None,
            gate=None, scale=1.0, res_scale=1.0, eps=1e-5):
    """x, res [R, C]. Returns y (None with pre "none"), the sum, stats [R, 4]."""
    x, res = _f64(x, res)
    R, C = x.shape
    w1, b1, w2, b2 = _params(C, post_weight, post_bias, pre_weight, pre_bias)
    stats = np.tile([0.0, 1.0, 0.0, 1.0], (R, 1))
    u = x
    if post != "none":
        u, stats[:, 0], stats[:, 1] = _norm(x, post, w1, b1, eps)
    s = scale * _gate_rows(gate, R, C) * u + (0.0 if res is None else res_scale * res)
    y = None
    if pre != "none":
        y, stats[:, 2], stats[:, 3] = _norm(s, pre, w2, b2, eps)
    return y, s, stats


def _norm_back(e, xh, rstd, kind):
    d = e - xh * (e * xh).mean(1, keepdims=True)
    return rstd[:, None] * (d - e.mean(1, keepdims=True) if kind == "layer" else d)


def addnorm_bwd(x, s, stats, dy=None, ds=None, pre="rms", pre_weight=None, pre_bias=None, post="none",
                post_weight=None, post_bias=None, gate=None, scale=1.0, res_scale=1.0):
    """Gradients at the sum s and the statistics that the call is given."""
    x, s, stats, dy, ds = _f64(x, s, stats, dy, ds)
    R, C = next(t for t in (x, s, dy) if t is not None).shape
    w1, b1, w2, b2 = _params(C, post_weight, post_bias, pre_weight, pre_bias)
    out = {}
    ds = np.zeros((R, C)) if ds is None else ds
    if pre != "none":
        xh = (s - stats[:, 2:3]) * stats[:, 3:4]
        out["dpre_weight"], out["dpre_bias"] = (dy * xh).sum(0), dy.sum(0)
        ds = ds + _norm_back(dy * w2, xh, stats[:, 3], pre)
    out["dres"] = res_scale * ds
    gr = _gate_rows(gate, R, C)
    du = scale * gr * ds
    if x is not None:
        xh = (x - stats[:, 0:1]) * stats[:, 1:2] if post != "none" else x
        if gate is not None:
            out["dgate"] = (scale * (xh * w1 + b1) * ds).reshape(len(gate), -1, C).sum(1)
    if post != "none":
        out["dpost_weight"], out["dpost_bias"] = (du * xh).sum(0), du.sum(0)
        du = _norm_back(du * w1, xh, stats[:, 1], post)
    out["dx"] = du
    return out


def rotary(x, inv_freq, positions, layout="half", scale=1.0, inverse=False):
    """x [B, L, H, W]; inv_freq [rot / 2]; positions [B, L]. The angle in the widest type that numpy has."""
    x = np.asarray(x, np.float64)
    rot = 2 * len(inv_freq)
    theta = np.asarray(positions, np.longdouble)[..., None] * np.asarray(inv_freq, np.longdouble)
    if inverse:
        theta = -theta
    c, s = (np.asarray(f(theta), np.float64)[:, :, None] * scale for f in (np.cos, np.sin))
    lo = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    hi = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    out = x.copy()
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., lo] * s + x[..., hi] * c
    return out
