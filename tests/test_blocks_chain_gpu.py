"""The operators of a residual network together, as they would be used: norm, gated recurrence, rotary positions,
linear attention, group norm, norm and sum; a prompt, its gradients by hand, and the same prompt token by token.

Tolerance: each of the six operators is within 2^9 roundings of 2^-24 of its terms' magnitudes, and sums of squares of
their errors add up; 2^12 roundings of the result's norm leave a factor of 3 for terms that cancel."""
import numpy as np
import pytest
import torch

from oracle import blocks as ref
from oracle import linattn as ref_la
from parity_util import to_np
from selective_state_space_48_amd import selscan as S

pytestmark = pytest.mark.gpu
ROOM = 2.0 ** -24 * 2 ** 12
B, L, H, W = 2, 45, 4, 16
C = H * W


def setup():
    g = torch.Generator().manual_seed(3)
    rn = lambda *s, std=1.0, m=0.0: (torch.randn(s, generator=g) * std + m).cuda()  # noqa: E731
    return dict(x=rn(B, L, C), res=rn(B, L, C), w_in=rn(C, std=0.2, m=1.0), Wg=rn(C, C, std=C ** -0.5),
                Wr=rn(C, C, std=C ** -0.5), Wz=rn(C, C, std=C ** -0.5), A=-0.3 * rn(C).abs(),
                inv=S.rotary_frequencies(W, device="cuda"),
                decay=torch.log1p(-(2.0 ** -torch.arange(3, 3 + H, dtype=torch.float32))).cuda(),
                gn_w=rn(C, std=0.2, m=1.0), w_post=rn(C, std=0.2, m=1.0), w_out=rn(C, std=0.2, m=1.0), b_out=rn(C))


def forward(p, x, res, at=0, gated=None, attend=None):
    """x, res [B, T, C]; `gated` and `attend` are the recurrence and the attention over T tokens."""
    T = x.shape[1]
    heads = lambda t: t.reshape(B, T, H, W)  # noqa: E731
    y0, r0, st0 = S.addnorm(x, res, pre_weight=p["w_in"])
    g, r, z = (y0 @ p[n] for n in ("Wg", "Wr", "Wz"))
    h = gated(y0, g, r, z)
    q, k = S.rotary(heads(h), heads(h), p["inv"], offset=at)
    y2 = attend(q, k, heads(h).contiguous())
    n, mean, rstd = S.groupnorm(y2.reshape(B * T, C), H, p["gn_w"])
    y3, r1, st1 = S.addnorm(n.reshape(B, T, C), r0, pre="layer", pre_weight=p["w_out"], pre_bias=p["b_out"],
                            post="rms", post_weight=p["w_post"], scale=0.5)
    return y3, r1, dict(y0=y0, r0=r0, st0=st0, g=g, r=r, z=z, h=h, q=q, k=k, y2=y2, mean=mean, rstd=rstd, n=n, st1=st1,
                        r1=r1)


def oracle(p, x, res):
    """The same chain in 64 bits."""
    flat = lambda t: t.reshape(B * L, C)  # noqa: E731
    y0, r0, _ = ref.addnorm(flat(x), flat(res), pre_weight=p["w_in"])
    y0 = y0.reshape(B, L, C)
    h, _, _ = ref.gated(y0, y0 @ p["Wg"], y0 @ p["Wr"], p["A"], y0 @ p["Wz"])
    pos = np.tile(np.arange(L), (B, 1))
    qk = ref.rotary(h.reshape(B, L, H, W), p["inv"], pos)
    y2, _ = ref_la.linattn(qk, qk, h.reshape(B, L, H, W), p["decay"])
    n, _, _ = ref_la.groupnorm(y2.reshape(B * L, 1, C), H, p["gn_w"], None, None, "none", 1e-5)
    y3, r1, _ = ref.addnorm(n.reshape(B * L, C), r0, pre="layer", pre_weight=p["w_out"], pre_bias=p["b_out"], post="rms",
                            post_weight=p["w_post"], scale=0.5)
    return y3.reshape(B, L, C), r1.reshape(B, L, C)


def prompt(p):
    return forward(p, p["x"], p["res"], 0, lambda y0, g, r, z: S.gated_fwd(y0, g, r, p["A"], z)[0],
                   lambda q, k, v: S.linattn_fwd(q, k, v, p["decay"])[0])


def near(got, want, what):
    got, want = to_np(got), np.asarray(want)
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    print(f"[parity] {what}: {off / ROOM:.3f} of the tolerance", flush=True)
    assert off <= ROOM, what


def test_prompt_and_gradients():
    print("[case] a layer's prompt and gradients", flush=True)
    p = setup()
    y3, r1, k = prompt(p)
    torch.cuda.synchronize()
    h = {n: to_np(t) for n, t in p.items()}
    wy, wr = oracle(h, h["x"], h["res"])
    near(y3, wy, "prompt y")
    near(r1, wr, "prompt residual")
    gen = torch.Generator().manual_seed(4)
    dy, dr = (torch.randn((B, L, C), generator=gen).cuda() for _ in range(2))
    # back through the chain
    b1 = S.addnorm_bwd(k["n"].reshape(B, L, C), k["r1"], dy=dy, dres_out=dr, stats=k["st1"], pre="layer",
                       pre_weight=p["w_out"], pre_bias=p["b_out"], post="rms", post_weight=p["w_post"], scale=0.5)
    gn = S.groupnorm_bwd(k["y2"].reshape(B * L, C), H, p["gn_w"], dy=b1["dx"].reshape(B * L, C), mean=k["mean"],
                         rstd=k["rstd"])
    v = k["h"].reshape(B, L, H, W)
    la = S.linattn_bwd(k["q"], k["k"], v, p["decay"], dy=gn["dx"].reshape(B, L, H, W))
    dq, dk = S.rotary(la["dq"], la["dk"], p["inv"], inverse=True)
    dh = (dq + dk + la["dv"]).reshape(B, L, C)
    ga = S.gated_bwd(k["y0"], k["g"], k["r"], p["A"], k["z"], dy=dh)
    dy0 = ga["dx"] + ga["dg"] @ p["Wg"].T + ga["dr"] @ p["Wr"].T + ga["dz"] @ p["Wz"].T
    b0 = S.addnorm_bwd(None, k["r0"], dy=dy0, dres_out=b1["dres"], stats=k["st0"], pre_weight=p["w_in"])
    torch.cuda.synchronize()
    assert torch.equal(b0["dx"], b0["dres"])  # x and res enter alike
    rng = np.random.default_rng(5)

    def loss(q):
        a, b = oracle(q, q["x"], q["res"])
        return (a * to_np(dy)).sum() + (b * to_np(dr)).sum()

    for name, got in (("x", b0["dx"]), ("res", b0["dres"]), ("A", ga["dA"]), ("w_in", b0["dpre_weight"]),
                      ("gn_w", gn["dweight"]), ("w_post", b1["dpost_weight"]), ("b_out", b1["dpre_bias"])):
        d = rng.standard_normal(h[name].shape) * (np.abs(h[name]) if name == "A" else 1.0)
        e = 1e-6
        diff = (loss(dict(h, **{name: h[name] + e * d})) - loss(dict(h, **{name: h[name] - e * d}))) / (2 * e)
        g = to_np(got)
        room = ROOM * np.linalg.norm(g) * np.linalg.norm(d) + 1e-5
        print(f"[parity] d{name}: {abs(diff - (g * d).sum()) / room:.3f} of the tolerance", flush=True)
        assert abs(diff - (g * d).sum()) <= room, name


def test_token_by_token():
    print("[case] the prompt token by token, captured in a graph", flush=True)
    p = setup()
    want, _, _ = prompt(p)
    torch.cuda.synchronize()
    state, kv = torch.zeros(B, C, device="cuda"), torch.zeros(B, H, W, W, device="cuda")
    one = lambda t: t[:, 0].contiguous()  # noqa: E731
    x, res = (torch.empty(B, 1, C, device="cuda") for _ in range(2))
    pos = torch.zeros(B, 1, dtype=torch.int32, device="cuda")

    def attend(q, k, v):
        return S.linattn_step(kv, one(q), one(k), one(v), p["decay"])[:, None]

    def token():
        T = 1
        heads = lambda t: t.reshape(B, T, H, W)  # noqa: E731
        y0, r0, _ = S.addnorm(x, res, pre_weight=p["w_in"])
        g, r, z = (y0 @ p[n] for n in ("Wg", "Wr", "Wz"))
        h = S.gated_step(state, one(y0), one(g), one(r), p["A"], one(z))[:, None]
        q, k = S.rotary(heads(h), heads(h), p["inv"], positions=pos)
        n, _, _ = S.groupnorm(attend(q, k, heads(h)).reshape(B, C), H, p["gn_w"])
        return S.addnorm(n.reshape(B, 1, C), r0, pre="layer", pre_weight=p["w_out"], pre_bias=p["b_out"], post="rms",
                         post_weight=p["w_post"], scale=0.5)[0]

    x.copy_(p["x"][:, :1])
    res.copy_(p["res"][:, :1])
    token()
    torch.cuda.synchronize()
    state.zero_()
    kv.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token()
    state.zero_()
    kv.zero_()
    got = []
    for t in range(L):
        x.copy_(p["x"][:, t:t + 1])
        res.copy_(p["res"][:, t:t + 1])
        pos.fill_(t)
        graph.replay()
        torch.cuda.synchronize()
        got.append(y.clone())
    near(torch.cat(got, 1), to_np(want), "tokens against the prompt")
