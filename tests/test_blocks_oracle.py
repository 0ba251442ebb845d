"""The 64-bit definitions of oracle/blocks.py against each other and against differences (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import blocks as ref

rng = np.random.default_rng(5)


def differences(loss, args, name, got):
    d = rng.standard_normal(args[name].shape) * np.minimum(np.abs(args[name]), 1)
    e = 1e-6
    diff = (loss(dict(args, **{name: args[name] + e * d})) - loss(dict(args, **{name: args[name] - e * d}))) / (2 * e)
    # rounding 2^-53 / e of sums below 2^8, and e^2 of third derivatives
    assert abs(diff - (got * d).sum()) <= 2.0 ** -53 * 256 / e * 8 + 1e-8, name


@pytest.mark.parametrize("decay", [False, True])
def test_gated_gradients(decay):
    B, L, D = 2, 9, 5
    a = {k: rng.standard_normal((B, L, D)) for k in ("x", "g", "z", "dy")}
    a.update(r=rng.standard_normal((B, L, D)) if decay else None, A=-rng.random(D) if decay else None,
             h0=rng.standard_normal((B, D)), dlast=rng.standard_normal((B, D)))
    lengths = [9, 4]

    def loss(p):
        y, last, _ = ref.gated(p["x"], p["g"], p["r"], p["A"], p["z"], p["h0"], lengths)
        return (y * p["dy"]).sum() + (last * p["dlast"]).sum()

    r = ref.gated_bwd(a["x"], a["g"], a["dy"], a["r"], a["A"], a["z"], a["h0"], lengths, a["dlast"])
    for n in ("x", "g", "z", "h0") + (("r", "A") if decay else ()):
        differences(loss, a, n, r["d" + n])


def test_mix_is_the_selective_scan():
    """Theorem 1 of "Mamba: Linear-Time Sequence Modeling with Selective State Spaces" (azimuth.plus): with N = 1,
    A = -1 and a step size of softplus(g), exp(delta A) = 1 - sigmoid(g). The scan's input term delta B x is the
    gate's with B = sigmoid(g) / delta (the scan's oracle has N = 16: the other states get B = 0)."""
    B, D, L = 2, 1, 12
    x, g = rng.standard_normal((B, D, L)), rng.standard_normal((B, D, L))
    delta = np.log1p(np.exp(g))
    Bm, Cm = np.zeros((B, 16, L)), np.zeros((B, 16, L))
    Bm[:, 0], Cm[:, 0] = (ref.sigmoid(g) / delta)[:, 0], 1.0
    f32 = np.float32
    got = oracle.fwd(x.astype(f32), g.astype(f32), -np.ones((D, 16), f32), Bm.astype(f32), Cm.astype(f32))
    want, _, _ = ref.gated(np.float64(x.astype(f32)).swapaxes(1, 2), np.float64(g.astype(f32)).swapaxes(1, 2))
    # B is rounded to fp32 on the way in: 2^-24 of sums of at most L terms
    assert np.abs(got["y"].swapaxes(1, 2) - want).max() <= 2.0 ** -23 * np.abs(x).max() * L


@pytest.mark.parametrize("post,pre", [("layer", "rms"), ("rms", "layer"), ("none", "rms"), ("layer", "none")])
def test_addnorm_gradients(post, pre):
    R, C, G = 6, 7, 2
    a = {k: rng.standard_normal((R, C)) for k in ("x", "res", "dy", "ds")}
    a.update({k: rng.standard_normal(C) for k in ("post_weight", "post_bias", "pre_weight", "pre_bias")})
    a["gate"] = rng.standard_normal((G, C))
    for n, kind in (("post", post), ("pre", pre)):
        if kind == "none":
            a[n + "_weight"] = a[n + "_bias"] = None
    kw = dict(post=post, pre=pre, scale=0.6, res_scale=1.7)
    names = ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")

    def loss(p):
        y, s, _ = ref.addnorm(p["x"], p["res"], **kw, **{k: p[k] for k in names})
        return (s * p["ds"]).sum() + (0 if y is None else (y * p["dy"]).sum())

    _, s, st = ref.addnorm(a["x"], a["res"], **kw, **{k: a[k] for k in names})
    r = ref.addnorm_bwd(a["x"], s, st, a["dy"] if pre != "none" else None, a["ds"], **kw, **{k: a[k] for k in names})
    for n in ("x", "res") + names:
        if a[n] is not None:
            differences(loss, a, n, r["d" + n])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary(layout):
    """Turns keep lengths, undo each other, and make products depend on the distance alone."""
    f = 10000.0 ** (-np.arange(0, 8, 2) / 8)
    q, k = rng.standard_normal((1, 1, 1, 10)), rng.standard_normal((1, 1, 1, 10))
    at = lambda x, p: ref.rotary(x, f, np.array([[p]]), layout)  # noqa: E731
    assert abs((at(q, 77) ** 2).sum() - (q ** 2).sum()) < 1e-13
    back = ref.rotary(at(q, 77), f, np.array([[77]]), layout, inverse=True)
    assert np.abs(back - q).max() < 1e-14
    assert abs((at(q, 30) * at(k, 12)).sum() - (at(q, 1018) * at(k, 1000)).sum()) < 1e-12
    assert (at(q, 5)[..., 8:] == q[..., 8:]).all()
