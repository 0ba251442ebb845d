"""Inputs, 64-bit references and tolerances of the linear-attention tests.

Tolerances are counted in roundings. An output is a sum of products; its scale
is the sum of the products' magnitudes (the oracle on the inputs' magnitudes).
Relative to that scale:
* fp32 sums: each term passes through at most L + dk + dv + 64 additions,
  each off by at most 2^-24;
* decays: powers of lambda, each formed with a handful of fp32 roundings
  (8 of 2^-24 for each hop over a chunk, at most L / 32 hops);
* bfloat16 calls: the operands of the matrix products are kept as two
  bfloat16 terms, off by at most 2^-8 * 2^-8 each, at most two of them in a
  product chain (a score or state operand, and a weighted operand).
The output's own rounding is half a step of its type, relative to the value.
"""
import numpy as np
import torch

from oracle import linattn as ref
from parity_util import to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def half(dtype):
    return torch.finfo(dtype).eps / 2


def relative(dtype, L, dk, dv):
    c = (L + dk + dv + 64) * 2.0 ** -24 + 8 * (L / 32 + 1) * 2.0 ** -24
    return c + (2 * 2.0 ** -16 if dtype == torch.bfloat16 else 0.0)


def close(got, want, scale, dtype, c, what):
    """|got - want| <= half a step of got's type (of the value it rounds) + c scale, everywhere."""
    got, want, scale = to_np(got), np.asarray(want), np.asarray(scale)
    assert got.shape == want.shape, f"{what}: {got.shape} {want.shape}"
    room = c * scale
    room = room + half(dtype) * (np.abs(want) + room) + 1e-37
    off = np.abs(got - want)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = float((off / room).max()) if off.size else 0.0
    print(f"[parity] {what}: {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def make(B, L, H, Hk, dk, dv, dtype, seed=0, h0=False, lengths=None, grads=False, device="cuda", decay=None):
    g = torch.Generator().manual_seed(seed)

    def rn(*s, dt=dtype):
        return torch.randn(s, generator=g).to(dt).to(device)

    p = dict(q=rn(B, L, H, dk), k=rn(B, L, Hk, dk), v=rn(B, L, Hk, dv))
    if decay is None:
        decay = torch.log1p(-(2.0 ** -(1 + 8 * torch.rand(H, generator=g))))
    p["log_decay"] = decay.float().to(device)
    p["h0"] = rn(B, H, dk, dv, dt=torch.float32) if h0 else None
    p["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=device)
    if grads:
        p["dy"] = rn(B, L, H, dv)
        p["dlast"] = rn(B, H, dk, dv, dt=torch.float32) if h0 else None
    return p


def host(p):
    return {k: None if t is None else to_np(t) for k, t in p.items()}


def fwd_ref(p, scale=None):
    h = host(p)
    n = h["lengths"]
    a = lambda x: None if x is None else np.abs(x)  # noqa: E731
    y, s = ref.linattn(h["q"], h["k"], h["v"], h["log_decay"], scale, h["h0"], n)
    ya, sa = ref.linattn(a(h["q"]), a(h["k"]), a(h["v"]), h["log_decay"], None if scale is None else abs(scale),
                         a(h["h0"]), n)
    return y, s, ya, sa


def bwd_ref(p, scale=None):
    h = host(p)
    a = lambda x: None if x is None else np.abs(x)  # noqa: E731
    args = [h[x] for x in ("q", "k", "v")]
    r = ref.linattn_bwd(*args, h["log_decay"], h["dy"], scale, h["h0"], h["lengths"], h["dlast"])
    s = ref.linattn_bwd(*map(a, args), h["log_decay"], a(h["dy"]), None if scale is None else abs(scale),
                        a(h["h0"]), h["lengths"], a(h["dlast"]))
    return r, s
