"""The norms around a block with the residual sum, and their gradients, on the GPU against the 64-bit definition.

Tolerances, in roundings U = 2^-24: sums over a row's C values pass through at most C / 64 + 64 additions each,
whose terms are formed with at most 16 roundings: c = (C / 64 + 80) U. An error in the mean shifts v - mean by that
share of the average |v|; rstd is off by half what the average square is, whose terms (v - mean)^2 are off by twice
their difference's error. What the first norm is off by enters the sum times gate and scale, and from there the
second norm's mean and square (by the averages of it). A column's sum passes through at most R additions. The
output's own rounding is half a step of its type."""
import numpy as np
import pytest
import torch

from blocks_util import DT, U, close
from oracle import blocks as ref
from parity_util import to_np
from selective_state_space_48_amd import selscan

pytestmark = pytest.mark.gpu
NORMS = ["none", "rms", "layer"]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]

SHAPES = [
    (1, 1), (3, 2), (5, 7), (2, 64), (9, 65), (4, 130), (33, 256), (7, 511), (130, 96), (3, 1000), (2, 2049), (5, 2560),
    (3, 4097), (2, 8192), (1, 12345), (3, 16384),
]


def case(msg):
    print(f"[case] {msg}", flush=True)


def make(R, C, types, seed=0, post="rms", pre="rms", gates=0, bias=True, weight=True, res=True, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    dt, rt = DT[types[0]], DT[types[1]]

    def rn(*s, dt=torch.float32, m=0.0):
        return (torch.randn(s, generator=g) + m).to(dt).cuda()

    p = dict(x=rn(R, C, dt=dt, m=mean), res=rn(R, C, dt=rt, m=mean) if res else None,
             gate=rn(gates, C) if gates else None)
    for n, kind in (("post", post), ("pre", pre)):
        there = kind != "none"
        p[n + "_weight"] = rn(C) if there and weight else None
        p[n + "_bias"] = rn(C) if there and bias else None
    p["dy"], p["ds"] = rn(R, C, dt=dt), rn(R, C, dt=rt)
    return p


def params(p, f=lambda t: t):
    return {k: None if p[k] is None else f(p[k]) for k in ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")}


def norm_room(v, dv, kind, w, b, mean, rstd, c):
    """Room of a norm of v (off by dv each): of the normed value, of the mean and of rstd (relative)."""
    av = np.abs(v)
    dm = (dv.mean(1) + c * av.mean(1) if kind == "layer" else np.zeros(len(v)))[:, None]
    r = rstd[:, None]
    d = np.abs(v - mean[:, None])
    dd = dv + dm + U * (d + av)
    dr = (d * dd).mean(1)[:, None] * r * r + c
    return np.abs(w) * r * (dd + d * dr) + 4 * U * (np.abs(w) * d * r + np.abs(b)), dm[:, 0], (dr * r)[:, 0]


def check(p, post, pre, what, scale=0.7, res_scale=1.3, eps=1e-5):
    R, C = p["x"].shape
    dt, rt = p["x"].dtype, p["ds"].dtype
    kw = dict(pre=pre, post=post, scale=scale, res_scale=res_scale)
    y, s, stats = selscan.addnorm(p["x"], p["res"], eps=eps, res_dtype=rt, **kw, **params(p))
    torch.cuda.synchronize()
    scale, res_scale = float(np.float32(scale)), float(np.float32(res_scale))
    kw.update(scale=scale, res_scale=res_scale)
    n = params(p, to_np)
    x, res = to_np(p["x"]), None if p["res"] is None else to_np(p["res"])
    wy, ws, wst = ref.addnorm(x, res, eps=eps, **kw, **n)
    w1, b1, w2, b2 = ref._params(C, n["post_weight"], n["post_bias"], n["pre_weight"], n["pre_bias"])
    c = (C / 64 + 80) * U
    gr = np.abs(ref._gate_rows(n["gate"], R, C) * scale)
    du, dm, dr = np.zeros((R, C)), np.zeros(R), np.zeros(R)
    u = x
    if post != "none":
        du, dm, dr = norm_room(x, np.zeros((R, C)), post, w1, b1, wst[:, 0], wst[:, 1], c)
        u = (x - wst[:, 0:1]) * wst[:, 1:2] * w1 + b1
    ds = gr * (du + 4 * U * np.abs(u)) + 2 * U * (0 if res is None else np.abs(res_scale * res))
    close(s, ws, ds, what + " res_out")
    dm2, dr2 = np.zeros(R), np.zeros(R)
    if pre != "none":
        dy, dm2, dr2 = norm_room(ws, ds, pre, w2, b2, wst[:, 2], wst[:, 3], c)
        close(y, wy, dy, what + " y")
    else:
        assert y is None
    close(stats, wst, np.stack((dm, dr, dm2, dr2), 1), what + " stats")

    ds_in = p["ds"]
    r = selscan.addnorm_bwd(p["x"], s if pre != "none" else None, dy=p["dy"] if pre != "none" else None,
                            dres_out=ds_in, stats=stats, **{**kw, **params(p)})
    torch.cuda.synchronize()
    want = ref.addnorm_bwd(x, to_np(s) if pre != "none" else None, to_np(stats),
                           to_np(p["dy"]) if pre != "none" else None, to_np(ds_in), **kw, **n)
    check_bwd(r, want, p, to_np(s), to_np(stats), post, pre, w1, b1, w2, gr, res_scale, c, what)
    return y, s, stats, r


def check_bwd(r, want, p, s, st, post, pre, w1, b1, w2, gr, res_scale, c, what):
    R, C = p["x"].shape
    x, dy, ds = (np.abs(to_np(p[k])) for k in ("x", "dy", "ds"))
    c = c + 16 * U
    avg = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    cc = (R + 64) * U

    def back(e, xh, rstd, kind):
        """magnitude of rstd (e - average(e) - xh average(e xh))"""
        return rstd * (e + (avg(e) if kind == "layer" else 0) + xh * avg(e * xh))

    mag, err = ds, np.zeros((R, C))
    if pre != "none":
        xh = (np.abs(s) + np.abs(st[:, 2:3])) * st[:, 3:4]
        e = dy * np.abs(w2)
        more = back(e, xh, st[:, 3:4], pre)
        mag, err = mag + more, more * c
        if "dpre_weight" in r:
            close(r["dpre_weight"], want["dpre_weight"], (dy * xh).sum(0) * (cc + c), what + " dpre_weight")
        if "dpre_bias" in r:
            close(r["dpre_bias"], want["dpre_bias"], dy.sum(0) * cc, what + " dpre_bias")
    err = err + 2 * U * mag
    close(r["dres"], want["dres"], abs(res_scale) * (err + 2 * U * mag), what + " dres")
    xh = (x + np.abs(st[:, 0:1])) * st[:, 1:2] if post != "none" else x
    if "dgate" in r:
        G = len(r["dgate"])
        u = xh * np.abs(w1) + np.abs(b1)
        sc = gr / np.maximum(np.abs(ref._gate_rows(to_np(p["gate"]), R, C)), 1e-30)
        room = (sc * u * (err + mag * (c + cc))).reshape(G, R // G, C).sum(1)
        close(r["dgate"], want["dgate"], room, what + " dgate")
    du, eu = gr * mag, gr * (err + 3 * U * mag)
    if post != "none":
        if "dpost_weight" in r:
            close(r["dpost_weight"], want["dpost_weight"], (xh * (eu + du * (cc + c))).sum(0), what + " dpost_weight")
        if "dpost_bias" in r:
            close(r["dpost_bias"], want["dpost_bias"], (eu + du * cc).sum(0), what + " dpost_bias")
        f = du * np.abs(w1)
        eu = back(eu * np.abs(w1), xh, st[:, 1:2], post) + c * back(f, xh, st[:, 1:2], post)
        du = back(f, xh, st[:, 1:2], post)
    close(r["dx"], want["dx"], eu + 2 * U * du, what + " dx")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, types):
    R, C = shape
    what = f"{shape} {types}"
    case(what)
    check(make(R, C, types, seed=1), "rms", "rms", what)
    check(make(R, C, types, seed=2, post="none", bias=False, res=False), "none", "layer", what + " plain")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("post", NORMS)
@pytest.mark.parametrize("pre", NORMS)
def test_norms(pre, post, types):
    for R, C, gates in ((12, 320, 0), (12, 320, 3), (6, 1111, 6), (6, 4096, 1)):
        what = f"post={post} pre={pre} {(R, C, gates)} {types}"
        case(what)
        check(make(R, C, types, seed=3, post=post, pre=pre, gates=gates, bias=gates != 1), post, pre, what)


def test_many_rows():
    """Rows over many workgroups, and gates whose rows end inside one's share."""
    for R, C, gates in ((5000, 64, 0), (3001, 40, 1), (1200, 513, 40), (700, 1024, 7), (20000, 8, 10)):
        what = f"{(R, C, gates)}"
        case(what)
        check(make(R, C, ("bf16", "bf16"), seed=4, post="layer", gates=gates), "layer", "rms", what)


@pytest.mark.parametrize("types", TYPES)
def test_wide_rows_with_gates(types):
    """Rows of more than 512 threads, whose sums over rows are formed in a launch of their own."""
    for R, C, gates in ((6, 9000, 0), (6, 9000, 2), (4, 16384, 1), (9, 8200, 9)):
        what = f"{(R, C, gates)} {types}"
        case(what)
        check(make(R, C, types, seed=14, post="layer", gates=gates), "layer", "rms", what)
    case("a gate without its gradient, sums without a gate")
    p = make(12, 9000, types, seed=15, post="none", gates=3)
    _, s, st = selscan.addnorm(p["x"], p["res"], gate=p["gate"], pre_weight=p["pre_weight"])
    r = selscan.addnorm_bwd(None, s, dy=p["dy"], stats=st, gate=p["gate"], pre_weight=p["pre_weight"],
                            want_dparams=False)
    full = selscan.addnorm_bwd(p["x"], s, dy=p["dy"], stats=st, gate=p["gate"], pre_weight=p["pre_weight"])
    torch.cuda.synchronize()
    assert sorted(r) == ["dres", "dx"] and all(torch.equal(r[k], full[k]) for k in r)


def test_many_gate_rows():
    """As many gate rows as workgroups, or more: each workgroup takes whole ones."""
    for R, C, gates in ((4000, 24, 2000), (3000, 600, 1500), (1024, 1000, 1024), (600, 9000, 300), (5000, 8, 5000)):
        what = f"{(R, C, gates)}"
        case(what)
        check(make(R, C, ("f32", "f32"), seed=16, post="rms", gates=gates, bias=False), "rms", "layer", what)


def test_far_mean_no_weights_other_eps():
    case("far mean")
    check(make(4, 700, ("f32", "f32"), seed=5, weight=False, bias=False, mean=300.0), "layer", "layer", "far mean",
          eps=0.1)


def test_constant_and_zero_rows():
    """No spread: the bias; rows of zeros: 0 with any eps above 0, gradients finite."""
    case("constant rows")
    x = torch.full((3, 96), 2.5, device="cuda")
    x[1] = 0
    b = torch.arange(96.0, device="cuda")
    y, s, stats = selscan.addnorm(x, None, pre="layer", pre_bias=b)
    r = selscan.addnorm_bwd(None, s, dy=torch.ones_like(x), stats=stats, pre="layer", pre_bias=b)
    y2, _, _ = selscan.addnorm(x, None, pre="rms")
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand(3, 96)) and all(torch.isfinite(t).all() for t in r.values())
    assert (y2[1] == 0).all()


@pytest.mark.parametrize("C", [33, 320, 2560, 5000])
def test_rows_do_not_meet(C):
    """A NaN stays in its row, and a row's result does not depend on the others."""
    case(f"rows {C}")
    p = make(40, C, ("bf16", "f32"), seed=6)
    kw = dict(post="rms", **params(p))
    y, s, st = selscan.addnorm(p["x"], p["res"], **kw)
    x2 = p["x"].clone()
    x2[7, C // 2] = float("nan")
    y2, s2, st2 = selscan.addnorm(x2, p["res"], **kw)
    y3, s3, st3 = selscan.addnorm(p["x"][11:12].clone(), p["res"][11:12].clone(), **kw)
    torch.cuda.synchronize()
    others = [i for i in range(40) if i != 7]
    assert torch.equal(y[others], y2[others]) and torch.equal(st[others], st2[others]) and torch.isnan(y2[7]).all()
    assert torch.equal(y[11:12], y3) and torch.equal(s[11:12], s3) and torch.equal(st[11:12], st3)


def test_in_place_and_options():
    case("in place, outputs that are not wanted, the caller's workspace")
    p = make(300, 640, ("bf16", "bf16"), seed=7, post="layer", gates=3)
    kw = dict(post="layer", **params(p))
    y, s, st = selscan.addnorm(p["x"], p["res"], **kw)
    res = p["res"].clone()
    y2, s2, none = selscan.addnorm(p["x"], res, **kw, res_out=res, return_stats=False)
    y3, s3, _ = selscan.addnorm(p["x"], p["res"], **kw, return_res=False)
    torch.cuda.synchronize()
    assert s2 is res and none is None and s3 is None
    assert torch.equal(y, y2) and torch.equal(s, res) and torch.equal(y, y3)
    bw = dict(dy=p["dy"], stats=st, **kw)
    r = selscan.addnorm_bwd(p["x"], s, dres_out=p["ds"], **bw)
    ds = p["ds"].clone()
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    r2 = selscan.addnorm_bwd(p["x"], s, dres_out=ds, dres=ds, workspace=ws, **bw)
    r3 = selscan.addnorm_bwd(p["x"], s, dres_out=p["ds"], want_dparams=False, want_dres=False, **bw)
    r4 = selscan.addnorm_bwd(p["x"], s, dres_out=p["ds"], want_dx=False, **bw)
    zeros = selscan.addnorm_bwd(p["x"], s, dres_out=torch.zeros_like(ds), **bw)
    left_out = selscan.addnorm_bwd(p["x"], s, **bw)
    torch.cuda.synchronize()
    assert r2["dres"] is ds and all(torch.equal(r[k], r2[k]) for k in r)
    assert sorted(r3) == ["dx"] and torch.equal(r["dx"], r3["dx"])
    assert "dx" not in r4 and all(torch.equal(r[k], r4[k]) for k in r4)
    assert all(torch.equal(zeros[k], left_out[k]) for k in zeros)


def test_leading_axes():
    case("leading axes")
    p = make(24, 128, ("f32", "f32"), seed=8)
    y, s, st = selscan.addnorm(p["x"], p["res"], pre_weight=p["pre_weight"])
    v = lambda t: t.reshape(2, 3, 4, 128)  # noqa: E731
    y2, s2, st2 = selscan.addnorm(v(p["x"]), v(p["res"]), pre_weight=p["pre_weight"])
    r = selscan.addnorm_bwd(None, s, dy=p["dy"], stats=st, pre_weight=p["pre_weight"])
    r2 = selscan.addnorm_bwd(None, s2, dy=v(p["dy"]), stats=st2, pre_weight=p["pre_weight"])
    torch.cuda.synchronize()
    assert torch.equal(v(y), y2) and torch.equal(v(s), s2) and torch.equal(st, st2)
    assert torch.equal(v(r["dx"]), r2["dx"]) and torch.equal(r["dpre_weight"], r2["dpre_weight"])


def test_empty():
    case("no rows, no channels")
    w = torch.ones(8, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    y, s, st = selscan.addnorm(x, x, pre_weight=w, gate=torch.ones(2, 8, device="cuda"))
    r = selscan.addnorm_bwd(x, s, dy=y, stats=st, pre_weight=w, gate=torch.ones(2, 8, device="cuda"))
    x0 = torch.empty(3, 0, device="cuda")
    _, _, st0 = selscan.addnorm(x0, x0, post="layer", eps=0.25)
    torch.cuda.synchronize()
    assert y.shape == (0, 8) and (r["dpre_weight"] == 0).all() and (r["dgate"] == 0).all()
    assert torch.equal(st0, torch.tensor([[0.0, 2.0, 0.0, 2.0]], device="cuda").expand(3, 4))


def test_gradients_against_differences():
    case("gradients against differences")
    rng = np.random.default_rng(9)
    R, C = 6, 50
    for post, pre in (("layer", "rms"), ("rms", "layer"), ("none", "rms"), ("rms", "none")):
        p = make(R, C, ("f32", "f32"), seed=10, post=post, pre=pre, gates=2)
        kw = dict(pre=pre, post=post, scale=0.5, res_scale=2.0)
        _, s, st = selscan.addnorm(p["x"], p["res"], **kw, **params(p))
        have = pre != "none"
        r = selscan.addnorm_bwd(p["x"], s if have else None, dy=p["dy"] if have else None, dres_out=p["ds"], stats=st,
                                **kw, **params(p))
        torch.cuda.synchronize()
        h = {k: None if t is None else to_np(t) for k, t in p.items()}

        def loss(b):
            y, s, _ = ref.addnorm(b["x"], b["res"], **kw, **params(b))
            return (s * h["ds"]).sum() + (0.0 if y is None else (y * h["dy"]).sum())

        for n in ("x", "res", "post_weight", "post_bias", "pre_weight", "pre_bias", "gate"):
            if h[n] is None:
                continue
            d = rng.standard_normal(h[n].shape)
            e = 1e-6
            diff = (loss(dict(h, **{n: h[n] + e * d})) - loss(dict(h, **{n: h[n] - e * d}))) / (2 * e)
            got = (to_np(r["d" + n]) * d).sum()
            # gradients within 300 roundings of terms that are below 5^4 (and their R rows' sums)
            room = 300 * U * 5 ** 4 * np.abs(d).sum() * (1 if n in ("x", "res") else R) + 1e-6
            assert abs(diff - got) <= room, (post, pre, n, diff, got, room)


@pytest.mark.parametrize("shape", [(64, 256), (20, 2560)])
def test_graph_and_streams(shape):
    R, C = shape
    case(f"graph and streams {shape}")
    p = make(R, C, ("bf16", "f32"), seed=11, gates=2)
    kw = dict(post="rms", **params(p))

    def both():
        y, s, st = selscan.addnorm(p["x"], p["res"], **kw)
        return {"y": y, "s": s, **selscan.addnorm_bwd(p["x"], s, dy=p["dy"], dres_out=p["ds"], stats=st, **kw)}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = both()
    torch.cuda.synchronize()
    want = both()
    torch.cuda.synchronize()
    assert all(torch.equal(on_side[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for turn in range(4):
        new = make(R, C, ("bf16", "f32"), seed=12 + turn, gates=2)
        for k in ("x", "res", "dy", "ds"):
            p[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in out.items()}
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want), turn
