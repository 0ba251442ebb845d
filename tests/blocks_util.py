"""Inputs and tolerances of the tests of the gated recurrence, in roundings of U = 2^-24.

Every bound is the first-order effect of the roundings that an fp32 evaluation
makes, carried through the recurrence with the magnitudes of its terms:
* sigmoid(v) and 1 - sigmoid(v): the exponent's argument is off by |v| U and the
  exponential, the sum, the reciprocal and the product by at most 8 U together:
  rho(v) = (2 |v| + 8) U, relative.
* a = exp(l), l = A sigmoid(r): a |l| (rho(r) + 4 U), and 8 U of the smaller of a
  and 1 - a for its evaluation; mix: rho(g) of the smaller of a and 1 - a.
* w = sqrt(1 - a^2): half the relative error of 1 - a, and 8 U; b: that, rho(g)
  and 4 U.
* a token's step: at most 4 U of the magnitude that the state can have.
The output's own rounding is half a step of its type, relative to the value.
"""
import numpy as np
import torch

from oracle import blocks as ref
from oracle.linattn import _lengths
from parity_util import to_np

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rho(v):
    return np.where(np.isinf(v), 8, 2 * np.where(np.isinf(v), 0, np.abs(v)) + 8) * U  # (of infinities: 0 or 1)


def np_of(p):
    return {k: (None if v is None else to_np(v)) if not isinstance(v, (int, float, str)) else v for k, v in p.items()}


def make(B, L, D, kind, dtype, seed=0, z=False, h0=False, lengths=None, grads=False, one=False, A=None, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def rn(*s, dt=dtype, std=1.0, mean=0.0):
        return (torch.randn(s, generator=g) * std + mean).to(dt).to(device)

    shape = (B, D) if one else (B, L, D)
    f32 = torch.float32
    p = dict(x=rn(*shape), g=rn(*shape, std=1.5), r=None, A=None, z=rn(*shape) if z else None, h0=None, lengths=None)
    if kind == "decay":
        p["r"] = rn(*shape, std=1.5)
        # rates from 2^-16 to 4: decays from hardly any to nearly all of it
        p["A"] = (-(2.0 ** (torch.rand(D, generator=g) * 18 - 16))).to(device) if A is None else A.to(device)
    if h0:
        p["h0"] = rn(B, D, dt=f32)
    if lengths is not None:
        p["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=device)
    if grads:
        p["dy"] = rn(*shape)
        p["dlast"] = rn(B, D, dt=f32) if h0 else None
    return p


def bounds(q):
    """The terms' absolute errors, the states' and the magnitudes they are measured with; q as np_of(make(...))."""
    a, c, w, b = ref.gated_terms(q["x"], q["g"], q["r"], q["A"])
    B, L, D = a.shape
    n = _lengths(q["lengths"], B, L)
    here = (np.arange(L) < n[:, None])[..., None]
    small = np.minimum(a, c)
    if q["r"] is None:
        da = small * rho(q["g"])
        dw = np.zeros_like(a)  # relative
        db = np.abs(b) * (rho(q["g"]) + 4 * U)
    else:
        l = np.abs(q["A"]) * ref.sigmoid(q["r"])
        da = a * l * 1.7 * (rho(q["r"]) + 4 * U) + small * 8 * U
        dw = np.divide(da, c, out=np.zeros_like(c), where=c > 0) + 8 * U
        db = np.abs(b) * (dw + rho(q["g"]) + 4 * U)
    a, b, da, db = (np.where(here, t, v) for t, v in ((a, 1.0), (b, 0.0), (da, 0.0), (db, 0.0)))
    h0 = None if q["h0"] is None else np.abs(q["h0"])
    H = np.zeros((B, D)) if h0 is None else h0
    E = H * U
    Hb, Eb, Ha, Ea = (np.empty((B, L, D)) for _ in range(4))
    for t in range(L):
        Hb[:, t], Eb[:, t] = H, E
        new = a[:, t] * H + np.abs(b[:, t])
        # (what enters a token counts too: the state is stepped from it)
        E = a[:, t] * E + da[:, t] * H + db[:, t] + np.where(here[:, t], 4 * U * new, 0.0)
        H = new
        Ha[:, t], Ea[:, t] = H, E
    return dict(a=a, c=c, w=w, b=b, da=da, dw=dw, Hb=Hb, Eb=Eb, Ha=Ha, Ea=Ea, H=H, E=E, here=here, n=n)


def close(got, want, room, what):
    """|got - want| <= half a step of got's type, of the value it rounds, + room, everywhere."""
    half = torch.finfo(got.dtype).eps / 2
    got, want = to_np(got), np.asarray(want)
    assert got.shape == want.shape, f"{what}: {got.shape} {want.shape}"
    room = np.broadcast_to(room, want.shape)
    room = room + half * (np.abs(want) + room) + 1e-37
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - want)
    worst = float((off / room).max()) if off.size else 0.0
    print(f"[parity] {what}: {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def check_fwd(y, last, q, what, ckpt=None):
    """The forward's outputs against the definition."""
    k = bounds(q)
    wy, wl, before = ref.gated(q["x"], q["g"], q["r"], q["A"], q["z"], q["h0"], q["lengths"])
    room, size = k["Ea"], k["Ha"]
    if q["z"] is not None:
        s = np.abs(ref.silu(q["z"]))
        room, size = room * s, size * s * (rho(q["z"]) / U + 4)
        room = room + size * U
    close(y, wy, np.where(k["here"], room, 0.0), what + " y")
    if last is not None:
        close(last, wl, k["E"], what + " last_state")
    if ckpt is not None:
        close(ckpt, before[:, ::64].swapaxes(0, 1), k["Eb"][:, ::64].swapaxes(0, 1), what + " ckpt")


def check_bwd(r, q, what):
    k = bounds(q)
    want = ref.gated_bwd(q["x"], q["g"], q["dy"], q["r"], q["A"], q["z"], q["h0"], q["lengths"], q["dlast"])
    x, g, here = np.abs(q["x"]), q["g"], k["here"]
    B, L, D = x.shape
    dy = np.where(here, np.abs(q["dy"]), 0.0)
    d, dd = dy, np.zeros_like(dy)
    if q["z"] is not None:
        s = np.abs(ref.silu(q["z"]))
        d, dd = dy * s, dy * s * (rho(q["z"]) + 4 * U)
    C = np.zeros((B, D)) if q["dlast"] is None else np.abs(q["dlast"])
    EC = C * U
    G, EG = np.empty((B, L, D)), np.empty((B, L, D))
    for t in range(L - 1, -1, -1):
        on = here[:, t]
        G[:, t], EG[:, t] = d[:, t] + C, dd[:, t] + EC + 2 * U * (d[:, t] + C)
        EC = np.where(on, k["a"][:, t] * EG[:, t] + k["da"][:, t] * G[:, t] + 4 * U * k["a"][:, t] * G[:, t], EC)
        C = np.where(on, k["a"][:, t] * G[:, t], C)
    v, w = ref.sigmoid(g), k["w"]
    vv = v * ref.sigmoid(-g)
    rg = rho(g)

    def c(name, room):
        close(r[name], want[name], np.where(here, room, 0.0), f"{what} {name}")

    f = w * v
    c("dx", f * EG + G * f * (k["dw"] + rg + 4 * U))
    if q["r"] is None:
        m = x + k["Hb"]
        c("dg", vv * (EG * m + G * (k["Eb"] + m * (2 * rg + 6 * U))))
    else:
        c("dg", w * x * vv * (EG + G * (k["dw"] + 2 * rg + 6 * U)))
        ratio = np.divide(k["a"], w, out=np.zeros_like(w), where=w > 0) * v * x
        K = k["Hb"] + ratio
        el = EG * k["a"] * K + G * k["da"] * K + G * k["a"] * (
            k["Eb"] + ratio * (k["dw"] + rg + 8 * U) + k["da"] / np.maximum(k["a"], 1e-30) * ratio + 4 * U * K)
        s, ml = ref.sigmoid(q["r"]), G * k["a"] * K
        rr = rho(q["r"])
        c("dr", np.abs(q["A"]) * s * ref.sigmoid(-q["r"]) * (el + ml * (2 * rr + 6 * U)))
        if "dA" in r:
            terms = np.where(here, s * ml, 0.0)
            room = np.where(here, s * (el + ml * (rr + 4 * U)), 0.0).sum((0, 1)) + terms.sum((0, 1)) * (B * L + 64) * U
            close(r["dA"], want["dA"], room, what + " dA")
    if q["z"] is not None:
        z = q["z"]
        c("dz", dy * (k["Ea"] * 1.1 + k["Ha"] * (1 + np.abs(z)) * (rho(z) + 8 * U)))
    if "dh0" in r:
        close(r["dh0"], want["dh0"], EC, what + " dh0")
