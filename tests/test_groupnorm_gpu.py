"""Group norm with an activation, channels last, and its gradients on the GPU
against the 64-bit definition; the chain it stands in (linear attention, norm,
gate, and back).

Tolerances, in roundings of 2^-24: sums over a group's n = S C / G values pass
through at most n / 256 + 64 additions each (fewer for small groups). An error
in the mean shifts x - mean by that share of the average |x|, so values and
averages are measured against xs = (|x| + average |x|) rstd, a bound of |xh|
and of how far its parts can cancel; exponentials, reciprocals and products
add at most 16 roundings, silu' another 16. The output's own rounding is half a
step of its type."""
import numpy as np
import pytest
import torch

from linattn_util import DT, bwd_ref, close, make
from oracle import linattn as ref
from parity_util import to_np
from selective_state_space_48_amd import selscan

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]
ACTS = ["none", "silu", "gate"]

SHAPES = [
    # (batch, spatial, channels, groups)
    (1, 1, 1, 1),
    (5, 1, 8, 8),          # one channel a group
    (7, 1, 30, 3),         # odd widths
    (33, 1, 256, 4),       # 64 channels a group
    (3, 1, 1024, 8),       # 128
    (300, 1, 64, 1),       # a plain row norm
    (2, 1, 5000, 2),       # long rows
    (1, 1, 16384, 4),
    (2, 7, 24, 3),
    (3, 65, 320, 32),      # 10 channels a group
    (2, 500, 64, 8),
    (1, 4099, 40, 5),      # many positions, an odd number
    (2, 1000, 512, 32),
    (1, 300, 2048, 1),     # one large group
    (70, 33, 96, 6),
    (3000, 1, 24, 3),      # column sums in two stages
    (700, 33, 40, 5),
    (2, 20000, 16, 2),     # many slabs
    (1, 3, 20000, 2),      # a row of a group wider than a workgroup
    (40, 1, 2560, 1),      # rows over several waves
]


def case(msg):
    print(f"[case] {msg}", flush=True)


def inputs(N, S, C, act, dtype, seed=0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, dt=dtype: torch.randn(s, generator=g).to(dt).cuda()  # noqa: E731
    shape = (N, C) if S == 1 else (N, S, C)
    p = dict(x=(torch.randn(shape, generator=g) * 1.5 + mean).to(dtype).cuda(), weight=rn(C, dt=torch.float32),
             bias=rn(C, dt=torch.float32), z=rn(*shape) if act == "gate" else None, dy=rn(*shape))
    return p


def check(p, N, S, C, G, act, what, eps=1e-5, affine=True):
    dt = p["x"].dtype
    w, b = (p["weight"], p["bias"]) if affine else (None, None)
    y, mean, rstd = selscan.groupnorm(p["x"], G, w, b, p["z"], act=act, eps=eps)
    torch.cuda.synchronize()
    x3 = to_np(p["x"]).reshape(N, S, C)
    z3 = None if p["z"] is None else to_np(p["z"]).reshape(N, S, C)
    wn, bn = (to_np(w), to_np(b)) if affine else (None, None)
    ry, rm, rr = ref.groupnorm(x3, G, wn, bn, z3, act, eps)
    n, D = S * C // G, C // G
    c = (n / 256 + 64) * 2.0 ** -24
    ax = np.abs(x3).reshape(N, S, G, D).mean((1, 3))
    per = lambda a: np.repeat(a, D, 1)[:, None]  # noqa: E731
    xs = (np.abs(x3) + per(ax)) * per(rr)
    # a relative error of rstd: half that of the variance, whose terms (x - mean)^2 are off by 2 |x - mean| c ax
    cr = c * (1 + (ax * rr))
    close(mean, rm, ax, torch.float32, c, what + " mean")
    close(rstd, rr, rr * (1 + ax * rr), torch.float32, c, what + " rstd")
    wa, ba = (np.abs(wn), np.abs(bn)) if affine else (1.0, 0.0)
    us = xs * wa * (1 + per(cr) / c) + ba
    gate = 1.1 * np.abs(z3) + 1e-30 if act == "gate" else 1.1
    close(y.reshape(N, S, C), ry, us * gate, dt, c + 16 * 2.0 ** -24, what + " y")

    r = selscan.groupnorm_bwd(p["x"], G, w, b, p["z"], act=act, dy=p["dy"], mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    dy3 = to_np(p["dy"]).reshape(N, S, C)
    want = ref.groupnorm_bwd(x3, G, wn, bn, z3, act, dy3, to_np(mean), to_np(rstd))
    xs = (np.abs(x3) + per(ax)) * per(to_np(rstd))
    us = xs * wa + ba
    # |silu'| <= 1.1 and |silu''| <= 0.5, so an error of u moves du by at most half of it
    da = np.abs(dy3) * (gate if act == "gate" else 1.1 + 0.5 * us if act == "silu" else 1.0)
    ea = da * wa
    avg = lambda a: per(a.reshape(N, S, G, D).mean((1, 3)))  # noqa: E731
    c = c + 32 * 2.0 ** -24
    close(r["dx"].reshape(N, S, C), want["dx"], per(to_np(rstd)) * (ea + avg(ea) + xs * avg(ea * xs)), dt, 2 * c,
          what + " dx")
    cc = c + (N * S / 64 + 64) * 2.0 ** -24
    close(r["dweight"], want["dweight"], (da * xs).sum((0, 1)), torch.float32, cc, what + " dweight")
    close(r["dbias"], want["dbias"], da.sum((0, 1)), torch.float32, cc, what + " dbias")
    if act == "gate":
        close(r["dz"].reshape(N, S, C), want["dz"], np.abs(dy3) * us * (1.1 + np.abs(z3)), dt, c, what + " dz")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_groupnorm(shape, dtype, act):
    N, S, C, G = shape
    case(f"groupnorm {shape} {dtype} {act}")
    check(inputs(N, S, C, act, DT[dtype], seed=1), N, S, C, G, act, f"{shape} {dtype} {act}")


@pytest.mark.parametrize("shape", [(4, 1, 512, 4), (2, 300, 64, 4)])
def test_far_mean_and_no_affine(shape):
    """A mean a thousand spreads away (the variance is not lost), without weight and bias, another eps."""
    N, S, C, G = shape
    case(f"far mean {shape}")
    check(inputs(N, S, C, "silu", torch.float32, seed=2, mean=1500.0), N, S, C, G, "silu", f"far {shape}", eps=0.1,
          affine=False)


def test_constant_groups():
    """No spread: y is the bias, the gradient of x is finite."""
    case("constant groups")
    x = torch.full((3, 64), 2.5, device="cuda")
    b = torch.arange(64.0, device="cuda")
    y, mean, rstd = selscan.groupnorm(x, 4, None, b)
    r = selscan.groupnorm_bwd(x, 4, None, b, dy=torch.ones_like(x), mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand(3, 64)) and (mean == 2.5).all() and torch.isfinite(r["dx"]).all()


def test_nan_stays_in_its_group():
    case("NaN in one group")
    p = inputs(4, 1, 256, "gate", torch.bfloat16, seed=3)
    p["x"][1, 70] = float("nan")
    y, mean, rstd = selscan.groupnorm(p["x"], 4, p["weight"], p["bias"], p["z"], act="gate")
    torch.cuda.synchronize()
    bad = torch.isnan(y)
    assert bad[1, 64:128].all() and bad.sum() == 64 and torch.isnan(mean).sum() == 1


def test_empty():
    case("no rows, no positions")
    w = torch.ones(8, device="cuda")
    for shape in ((0, 8), (2, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd = selscan.groupnorm(x, 2, w, w, act="silu", eps=0.25)
        r = selscan.groupnorm_bwd(x, 2, w, w, act="silu", dy=x, mean=mean, rstd=rstd)
        torch.cuda.synchronize()
        assert y.shape == shape and (mean == 0).all() and (rstd == 2).all()
        assert (r["dweight"] == 0).all() and (r["dbias"] == 0).all()


@pytest.mark.parametrize("shape", [(300, 1, 512, 4), (2, 700, 96, 6)])
def test_deterministic_workspace_and_options(shape):
    N, S, C, G = shape
    case(f"determinism, the caller's workspace {shape}")
    p = inputs(N, S, C, "gate", torch.bfloat16, seed=4)
    kw = dict(weight=p["weight"], bias=p["bias"], z=p["z"], act="gate")
    y, mean, rstd = selscan.groupnorm(p["x"], G, **kw)
    r = selscan.groupnorm_bwd(p["x"], G, **kw, dy=p["dy"], mean=mean, rstd=rstd)
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    y2, m2, s2 = selscan.groupnorm(p["x"], G, **kw, workspace=ws)
    r2 = selscan.groupnorm_bwd(p["x"], G, **kw, dy=p["dy"], mean=mean, rstd=rstd, workspace=ws)
    y3, m3, _ = selscan.groupnorm(p["x"], G, **kw, return_stats=False)
    r3 = selscan.groupnorm_bwd(p["x"], G, **kw, dy=p["dy"], mean=mean, rstd=rstd, want_dweight=False, want_dbias=False)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(mean, m2) and torch.equal(rstd, s2)
    assert all(torch.equal(r[n], r2[n]) for n in r)
    assert torch.equal(y, y3) and m3 is None
    assert sorted(r3) == ["dx", "dz"] and all(torch.equal(r[n], r3[n]) for n in r3)


def test_gradients_against_differences():
    N, S, C, G = 3, 40, 24, 3
    case("gradients against differences")
    rng = np.random.default_rng(6)
    for act in ACTS:
        p = inputs(N, S, C, act, torch.float32, seed=5)
        y, mean, rstd = selscan.groupnorm(p["x"], G, p["weight"], p["bias"], p["z"], act=act)
        r = selscan.groupnorm_bwd(p["x"], G, p["weight"], p["bias"], p["z"], act=act, dy=p["dy"], mean=mean, rstd=rstd)
        h = {k: None if t is None else to_np(t) for k, t in p.items()}

        def loss(b):
            return (ref.groupnorm(b["x"], G, b["weight"], b["bias"], b["z"], act)[0] * h["dy"]).sum()

        for n in ("x", "weight", "bias", "z"):
            if h[n] is None:
                continue
            d = rng.standard_normal(h[n].shape)
            e = 1e-6
            diff = (loss(dict(h, **{n: h[n] + e * d})) - loss(dict(h, **{n: h[n] - e * d}))) / (2 * e)
            got = (to_np(r["d" + n]) * d).sum()
            # every gradient within 100 roundings of terms no larger than |dy| (|x|, |z|, |w| <= 5) sums
            room = 200 * 2.0 ** -24 * 5 ** 3 * np.abs(d).sum() * np.abs(h["dy"]).max() * (1 if n in "xz" else N * S)
            assert abs(diff - got) <= room, (act, n, diff, got, room)


@pytest.mark.parametrize("shape", [(64, 1, 256, 4), (2, 600, 64, 4)])
def test_graph_and_streams(shape):
    N, S, C, G = shape
    case(f"graph and streams {shape}")
    p = inputs(N, S, C, "gate", torch.bfloat16, seed=7)

    def both():
        kw = dict(weight=p["weight"], bias=p["bias"], z=p["z"], act="gate")
        y, mean, rstd = selscan.groupnorm(p["x"], G, **kw)
        return {"y": y, **selscan.groupnorm_bwd(p["x"], G, **kw, dy=p["dy"], mean=mean, rstd=rstd)}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = both()
    torch.cuda.synchronize()
    want = both()
    torch.cuda.synchronize()
    assert all(torch.equal(on_side[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for turn in range(4):
        new = inputs(N, S, C, "gate", torch.bfloat16, seed=8 + turn)
        for k in ("x", "z", "dy"):
            p[k].copy_(new[k])
        g.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in out.items()}
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want), turn


def test_offsets_past_2_31():
    """More than 2^31 elements: the last rows, against a call on them alone."""
    N, C, G = 540000, 4096, 32
    case(f"offsets past 2^31: {N} x {C}")
    g = torch.Generator(device="cuda").manual_seed(9)
    x, dy = (torch.empty((N, C), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    assert x.numel() > 2 ** 31
    w = torch.ones(C, device="cuda")
    y, mean, rstd = selscan.groupnorm(x, G, w, act="silu")
    r = selscan.groupnorm_bwd(x, G, w, act="silu", dy=dy, mean=mean, rstd=rstd)
    xs = x[-70:].contiguous()
    y1, m1, s1 = selscan.groupnorm(xs, G, w, act="silu")
    r1 = selscan.groupnorm_bwd(xs, G, w, act="silu", dy=dy[-70:].contiguous(), mean=m1, rstd=s1)
    torch.cuda.synchronize()
    assert torch.equal(y[-70:], y1) and torch.equal(mean[-70:], m1) and torch.equal(r["dx"][-70:], r1["dx"])


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_chain(dtype):
    """The layer as it is used: heads, each normalised by itself, gated; and the gradients back through
    both. Every call is compared with the definition at the values that it was given."""
    B, L, H, Hk, d = 2, 70, 4, 2, 64
    case(f"chain {dtype}")
    p = make(B, L, H, Hk, d, d, DT[dtype], seed=10, grads=True, lengths=[70, 33])
    g = torch.Generator().manual_seed(11)
    z, dy = ((torch.randn((B * L, H * d), generator=g) + 0.3).to(DT[dtype]).cuda() for _ in range(2))
    w = torch.randn(H * d, generator=g).cuda()
    o, _ = selscan.linattn_fwd(p["q"], p["k"], p["v"], p["log_decay"], lengths=p["lengths"])
    flat = o.view(B * L, H * d)
    q = dict(x=flat, weight=w, bias=torch.zeros_like(w), z=z, dy=dy)
    check(q, B * L, 1, H * d, H, "gate", f"chain {dtype}")
    y, mean, rstd = selscan.groupnorm(flat, H, w, None, z, act="gate")
    r = selscan.groupnorm_bwd(flat, H, w, None, z, act="gate", dy=dy, mean=mean, rstd=rstd)
    p["dy"] = r["dx"].view(B, L, H, d)
    gr = selscan.linattn_bwd(p["q"], p["k"], p["v"], p["log_decay"], dy=p["dy"], lengths=p["lengths"])
    torch.cuda.synchronize()
    assert (y.view(B, L, H * d)[1, 33:] == 0).all()  # a padded token: all groups 0, and no bias
    want, size = bwd_ref(p)
    from linattn_util import relative
    for n in gr:
        close(gr[n], want[n], size[n], gr[n].dtype, relative(DT[dtype], L + 78, d, d), f"chain {dtype} {n}")


@pytest.mark.parametrize("shape", [(131072, 2, 512, 512), ((1 << 21) + 77, 1, 1025, 1)])
def test_many_entries(shape):
    """Many entries of many small groups, and more rows of wide groups than workgroups: the last entries
    against a call on them alone, the column sums against 64 bits."""
    N, S, C, G = shape
    case(f"many entries {shape}")
    g = torch.Generator(device="cuda").manual_seed(12)
    full = (N, C) if S == 1 else (N, S, C)
    x, dy = (torch.empty(full, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.ones(C, device="cuda")
    y, mean, rstd = selscan.groupnorm(x, G, w)
    r = selscan.groupnorm_bwd(x, G, w, dy=dy, mean=mean, rstd=rstd)
    last = x[-70:].clone(), dy[-70:].clone()  # (a view of odd rows would not be aligned)
    y1, m1, s1 = selscan.groupnorm(last[0], G, w)
    r1 = selscan.groupnorm_bwd(last[0], G, w, dy=last[1], mean=m1, rstd=s1)
    torch.cuda.synchronize()
    assert torch.equal(y[-70:], y1) and torch.equal(mean[-70:], m1) and torch.equal(rstd[-70:], s1)
    assert torch.equal(r["dx"][-70:], r1["dx"])
    want = {n: torch.zeros(C, dtype=torch.float64, device="cuda") for n in ("dweight", "dbias", "sw", "sb")}
    for a in range(0, N, 1 << 17):
        part = slice(a, a + (1 << 17))
        per = lambda t: t[part].double().repeat_interleave(C // G, 1)[:, None]  # noqa: E731
        d = dy[part].double().reshape(-1, S, C)
        t = d * (x[part].double().reshape(-1, S, C) - per(mean)) * per(rstd)
        for n, v in (("dweight", t), ("dbias", d), ("sw", t.abs()), ("sb", d.abs())):
            want[n] += v.sum((0, 1))
    # at most N S / 64 + 64 additions each and 8 roundings of a term, either way alike: six times their root
    c = 6 * (N * S / 64 + 72) ** 0.5 * 2.0 ** -24
    close(r["dweight"], to_np(want["dweight"]), to_np(want["sw"]), torch.float32, c, f"many entries {shape} dweight")
    close(r["dbias"], to_np(want["dbias"]), to_np(want["sb"]), torch.float32, c, f"many entries {shape} dbias")


def test_wide_groups_over_many_positions():
    """80000 values a thread, with an offset: the statistics and the averages of the gradients. In roundings
    of 2^-24: a workgroup's sum of its threads' is 6 + 16 additions, and 8 more for an average, a root, a
    quotient and the difference that a term is; not what the threads' own sums pass through."""
    N, S, C = 1, 40000, 2051
    case(f"wide groups over many positions {N, S, C}")
    g = torch.Generator(device="cuda").manual_seed(13)
    x = torch.randn((N, S, C), device="cuda", generator=g).add_(3.0)
    dy = torch.randn((N, S, C), device="cuda", generator=g).add_(x, alpha=0.5)
    y, mean, rstd = selscan.groupnorm(x, 1)
    r = selscan.groupnorm_bwd(x, 1, dy=dy, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    c = 30 * 2.0 ** -24
    xd = x.double()
    m, v = xd.mean(), xd.var(correction=0) + 1e-5
    for what, got, want in (("mean", mean, m), ("rstd", rstd, v.rsqrt())):
        off = abs(got.double().item() / want.item() - 1)
        print(f"[parity] wide groups {what}: {off * 2 ** 24:.2f} roundings", flush=True)
        assert off <= c, what
    xh, e = xd.sub_(mean.double()).mul_(rstd.double()), dy.double()
    m1, m2 = e.mean(), (e * xh).mean()
    want = (e - m1 - xh * m2) * rstd.double()
    room = (e.abs() + m1.abs() + xh.abs() * m2.abs()) * rstd.double() * c
    worst = ((r["dx"].double() - want).abs() / room).max().item()
    print(f"[parity] wide groups dx: {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1


@pytest.mark.parametrize("shape,dtype,act", [((8300, 1, 4096, 32), "bf16", "gate"), ((8300, 1, 4096, 4), "bf16", "silu"),
                                             ((4200, 1, 4096, 32), "f32", "none"), ((4200, 1, 4096, 4), "f32", "gate")])
def test_outputs_past_the_caches(shape, dtype, act):
    """Rows whose output is above 64 MB, which is stored past the caches, against the definition, with the
    sums over so many rows."""
    N, S, C, G = shape
    case(f"outputs past the caches {shape} {dtype} {act}")
    assert N * C * (2 if dtype == "bf16" else 4) > 64 << 20
    check(inputs(N, S, C, act, DT[dtype], seed=14), N, S, C, G, act, f"{shape} {dtype} {act}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 700, 2055, 1), (3, 5, 16400, 2), (1, 40, 33000, 2)])
def test_wide_groups(shape, dtype, act):
    """Groups wider than a workgroup's vectors, over few and many positions."""
    N, S, C, G = shape
    case(f"wide groups {shape} {dtype} {act}")
    check(inputs(N, S, C, act, DT[dtype], seed=15, mean=2.0), N, S, C, G, act, f"{shape} {dtype} {act}")
