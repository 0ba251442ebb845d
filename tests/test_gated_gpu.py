"""The gated linear recurrence on the GPU (prompts, single tokens, gradients)
against the 64-bit definition; tolerances as derived in blocks_util."""
import numpy as np
import pytest
import torch

from blocks_util import DT, U, bounds, check_bwd, check_fwd, close, make, np_of, rho
from oracle import blocks as ref
from parity_util import to_np
from selective_state_space_48_amd import selscan

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]
KINDS = ["mix", "decay"]

SHAPES = [
    # (batch, tokens, channels)
    (1, 1, 1),
    (2, 1, 64),
    (1, 2, 3),
    (3, 7, 33),
    (1, 63, 64),
    (2, 64, 65),
    (1, 65, 130),
    (2, 127, 100),
    (1, 128, 64),
    (1, 129, 7),
    (2, 300, 96),
    (1, 1000, 62),
    (5, 513, 31),
    (1, 2051, 16),
    (1, 70, 16384),  # channels enough for wide workgroups
    (1, 200, 8200),
]


def case(msg):
    print(f"[case] {msg}", flush=True)


def forward(p, ckpt=False, **kw):
    B, L, D = p["x"].shape
    c = torch.full(selscan.gated_ckpt_shape(B, L, D), float("nan"), device="cuda") if ckpt else None
    y, last = selscan.gated_fwd(p["x"], p["g"], p["r"], p["A"], p["z"], h0=p["h0"], lengths=p["lengths"], ckpt=c, **kw)
    torch.cuda.synchronize()
    return y, last, c


def backward(p, ckpt=None, **kw):
    r = selscan.gated_bwd(p["x"], p["g"], p["r"], p["A"], p["z"], dy=p["dy"], h0=p["h0"], lengths=p["lengths"],
                          dlast_state=p["dlast"], ckpt=ckpt, want_dh0=True, **kw)
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_fwd_bwd(shape, dtype, kind):
    B, L, D = shape
    for z, h0 in ((False, False), (True, True)):
        what = f"{shape} {dtype} {kind} z={z} h0={h0}"
        case(what)
        p = make(B, L, D, kind, DT[dtype], seed=1, z=z, h0=h0, grads=True)
        q = np_of(p)
        y, last, c = forward(p, ckpt=True)
        check_fwd(y, last, q, what, c)
        check_bwd(backward(p, c), q, what + " ckpt")
        check_bwd(backward(p), q, what)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_lengths(dtype, kind):
    """Padded batches: lengths of nothing, of one token, at and around tiles, past the end and below 0; what
    stands behind them is not read and comes out as zeros."""
    L, D = 300, 70
    lengths = [0, 1, 63, 64, 65, 128, 299, 300, 1000, -5]
    case(f"lengths {dtype} {kind}")
    p = make(len(lengths), L, D, kind, DT[dtype], seed=2, z=True, h0=True, lengths=lengths, grads=True)
    q = np_of(p)
    for b, n in enumerate(lengths):
        for k in ("x", "g", "r", "z", "dy"):
            if p[k] is not None:
                p[k][b, max(n, 0):] = float("nan")
    for segments in (0, 3):
        y, last, c = forward(p, ckpt=True, segments=segments)
        what = f"lengths {dtype} {kind} segments={segments}"
        check_fwd(y, last, q, what, c)
        check_bwd(backward(p, c, segments=segments), q, what + " ckpt")
        check_bwd(backward(p, segments=segments), q, what)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("segments", [1, 2, 5, 64])
def test_segments(segments, kind):
    """Runs of tokens in parallel, more of them than tiles too."""
    for B, L, D in ((1, 1500, 40), (2, 700, 130)):
        p = make(B, L, D, kind, torch.float32, seed=3, z=True, h0=True, grads=True)
        what = f"segments={segments} {(B, L, D)} {kind}"
        case(what)
        q = np_of(p)
        y, last, c = forward(p, ckpt=True, segments=segments)
        check_fwd(y, last, q, what, c)
        check_bwd(backward(p, c, segments=segments), q, what + " ckpt")
        check_bwd(backward(p, segments=segments), q, what)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_steps_equal_prompt(dtype, kind):
    """Single tokens against the definition, and a prompt's tokens one by one, each from the last one's state."""
    B, L, D = 5, 6, 131
    case(f"steps {dtype} {kind}")
    p = make(B, L, D, kind, DT[dtype], seed=4, z=True, h0=True)
    q = np_of(p)
    k = bounds(q)
    wy, wl, _ = ref.gated(q["x"], q["g"], q["r"], q["A"], q["z"], q["h0"])
    state = p["h0"].clone()
    for t in range(L):
        at = {n: None if p[n] is None else p[n][:, t].contiguous() for n in ("x", "g", "r", "z")}
        y = selscan.gated_step(state, at["x"], at["g"], at["r"], p["A"], at["z"])
        torch.cuda.synchronize()
        s = np.abs(ref.silu(q["z"][:, t]))
        close(y, wy[:, t], k["Ea"][:, t] * s + k["Ha"][:, t] * s * (rho(q["z"][:, t]) + 4 * U), f"step {t}")
    close(state, wl, k["E"], "state after the steps")


@pytest.mark.parametrize("kind", KINDS)
def test_split_sequence(kind):
    """A sequence in two pieces, the state handed on in place, and its gradients handed back."""
    B, L, D, cut = 2, 333, 66, 150
    case(f"split {kind}")
    p = make(B, L, D, kind, torch.float32, seed=5, h0=True, grads=True)
    q = np_of(p)
    part = lambda a, b: {k: v[:, a:b].contiguous() if v is not None and v.dim() == 3 else v for k, v in p.items()}  # noqa: E731
    p1, p2 = part(0, cut), part(cut, L)
    state = p["h0"].clone()
    y1, _ = selscan.gated_fwd(p1["x"], p1["g"], p1["r"], p1["A"], h0=state, last_state=state)
    mid = state.clone()
    y2, _ = selscan.gated_fwd(p2["x"], p2["g"], p2["r"], p2["A"], h0=state, last_state=state, segments=2)
    check_fwd(torch.cat((y1, y2), 1), state, q, f"split {kind}")
    p2["h0"] = mid
    r2 = backward(p2)
    p1["dlast"] = r2["dh0"]
    r1 = backward(p1)
    r = {k: torch.cat((r1[k], r2[k]), 1) for k in r1 if r1[k].dim() == 3}
    r["dh0"] = r1["dh0"]
    check_bwd(r, q, f"split {kind}")


def test_long_memory_keeps_what_it_settles_to():
    """A constant input through decays of 1 - 2^-8 to 1 - 2^-20: what 1 - a rounds to would show as a state off by
    up to 2^-5, a state stepped in 32 bits as one that stops short of where it goes."""
    case("long memory")
    L, D = 40000, 64
    A = -(2.0 ** -torch.linspace(8, 20, D)).cuda()
    x = torch.ones(1, L, D, device="cuda")
    g, r = torch.zeros_like(x), torch.full_like(x, 40.0)  # sigmoid(r) rounds to 1
    y, last = selscan.gated_fwd(x, g, r, A)
    torch.cuda.synchronize()
    l = to_np(A)
    b = np.sqrt(-np.expm1(2 * l)) * 0.5
    want = b * np.expm1(l * L) / np.expm1(l)
    # e and b to 32 roundings each; the sums within a tile of 16 tokens or so to 16
    close(last[0], want, np.abs(want) * 96 * U, "long memory")
    close(y[0, -1], want, np.abs(want) * 96 * U, "long memory y")


def test_reset_forgets():
    """A decay of 0 forgets a state of any size; one of nearly 0 leaves its share, to fp32 accuracy."""
    case("reset")
    for kind in KINDS:
        p = make(2, 40, 33, kind, torch.float32, seed=6, h0=True)
        p["h0"] = p["h0"] * 1e20
        if kind == "mix":
            p["g"][0, 5], p["g"][1, 20] = float("inf"), 30.0
        else:
            p["A"] = torch.full_like(p["A"], -60.0)
            p["r"][0, 5], p["r"][1, 20] = 5.0, 2.0
        y, last, _ = forward(p)
        check_fwd(y, last, np_of(p), f"reset {kind}")


def test_extreme_gates():
    """Gates of +-100 and infinities, and rates of 0: decays and weights of exactly 0 and 1, finite gradients."""
    case("extreme gates")
    for kind in KINDS:
        p = make(2, 70, 40, kind, torch.float32, seed=7, z=True, h0=True, grads=True)
        for n in ("g", "r", "z"):
            if p[n] is not None:
                for i, v in enumerate((100.0, -100.0, 300.0, -300.0, 60.0, -60.0)):
                    p[n][:, i::11, i::3] = v
        if kind == "decay":
            p["A"][::5] = 0.0
            p["A"][1::5] = -500.0
        q = np_of(p)
        y, last, c = forward(p, ckpt=True)
        check_fwd(y, last, q, f"extreme {kind}", c)
        r = backward(p, c)
        assert all(torch.isfinite(t).all() for t in r.values())
        if kind == "mix":
            check_bwd(r, q, f"extreme {kind}")


@pytest.mark.parametrize("segments", [1, 4])
def test_what_is_not_finite_stays_in_its_channel_and_after(segments):
    case("not finite")
    for kind in KINDS:
        p = make(2, 500, 70, kind, torch.bfloat16, seed=8, grads=True)
        clean, _, _ = forward(p, segments=segments)
        p["x"][1, 203, 17] = float("nan")
        p["x"][0, 77, 68] = float("inf")
        y, last, _ = forward(p, segments=segments)
        same = torch.ones_like(y, dtype=torch.bool)
        same[1, 203:, 17] = same[0, 77:, 68] = False
        assert torch.equal(y[same], clean[same]) and torch.isnan(y[1, 203:, 17]).all()
        assert torch.isnan(last[1, 17]) and torch.isfinite(last[1, :17]).all()
        if kind == "decay":
            p["A"][3] = 0.5  # no sqrt(1 - a^2)
            y, _, _ = forward(p, segments=segments)
            assert torch.isnan(y[:, :, 3]).all() and torch.isfinite(y[:, :, 4:17]).all()


def test_deterministic_workspace_and_options():
    case("determinism, the caller's workspace")
    p = make(2, 900, 200, "decay", torch.bfloat16, seed=9, z=True, h0=True, grads=True)
    y, last, c = forward(p, ckpt=True, segments=3)
    r = backward(p, c, segments=3)
    ws = torch.full((8 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    y2, last2, c2 = forward(p, ckpt=True, segments=3, workspace=ws)
    r2 = backward(p, c, segments=3, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(c, c2)
    assert all(torch.equal(r[k], r2[k]) for k in r)
    y3, last3 = selscan.gated_fwd(p["x"], p["g"], p["r"], p["A"], p["z"], h0=p["h0"], return_last_state=False, segments=3)
    r3 = selscan.gated_bwd(p["x"], p["g"], p["r"], p["A"], p["z"], dy=p["dy"], h0=p["h0"], dlast_state=p["dlast"],
                           ckpt=c, want_dA=False, segments=3)
    torch.cuda.synchronize()
    assert last3 is None and torch.equal(y, y3) and sorted(r3) == ["dg", "dr", "dx", "dz"]
    assert all(torch.equal(r[k], r3[k]) for k in r3)
    need = selscan.gated_bwd_workspace_size(2, 900, 200, torch.bfloat16, segments=3)
    with pytest.raises(selscan.SelscanError):
        backward(p, segments=3, workspace=ws[:need - 256])


def test_empty():
    case("no tokens, no channels, no entries")
    for shape in ((2, 0, 8), (0, 5, 8), (2, 5, 0)):
        B, L, D = shape
        p = make(B, L, D, "decay", torch.float32, seed=10, h0=True, grads=True)
        y, last, c = forward(p, ckpt=True)
        r = backward(p, c)
        assert y.shape == shape and torch.equal(last, p["h0"])
        assert torch.equal(r["dh0"], p["dlast"]) and (r["dA"] == 0).all()
    st = torch.empty(0, 8, device="cuda")
    assert selscan.gated_step(st, st, st).shape == (0, 8)


def test_gradients_against_differences():
    case("gradients against differences")
    rng = np.random.default_rng(11)
    for kind in KINDS:
        p = make(2, 50, 24, kind, torch.float32, seed=11, z=True, h0=True, lengths=[50, 31], grads=True)
        q = np_of(p)
        _, _, c = forward(p, ckpt=True)
        r = backward(p, c)

        def loss(b):
            y, last, _ = ref.gated(b["x"], b["g"], b["r"], b["A"], b["z"], b["h0"], b["lengths"])
            return (y * b["dy"]).sum() + (last * b["dlast"]).sum()

        for n in ("x", "g", "r", "A", "z", "h0"):
            if q[n] is None:
                continue
            d = rng.standard_normal(q[n].shape) * (np.abs(q[n]) if n == "A" else 1.0)
            e = 1e-6
            diff = (loss(dict(q, **{n: q[n] + e * d})) - loss(dict(q, **{n: q[n] - e * d}))) / (2 * e)
            got = (to_np(r["d" + n]) * d).sum()
            # every gradient within some 400 roundings of terms below 2^7 in sum (|dy|, |x|, |z|, |h| below 5)
            room = 400 * U * 2 ** 7 * np.abs(d).sum() * (50 if n == "A" else 1) + 1e-6
            assert abs(diff - got) <= room, (kind, n, diff, got, room)


@pytest.mark.parametrize("kind", KINDS)
def test_graph_and_streams(kind):
    """Captured with its gradients, replayed over new inputs with eager work between; on a side stream."""
    case(f"graph and streams {kind}")
    B, L, D = 2, 1100, 96
    p = make(B, L, D, kind, torch.bfloat16, seed=12, z=True, h0=True, grads=True)
    ck = torch.empty(selscan.gated_ckpt_shape(B, L, D), device="cuda")

    def both():
        y, last = selscan.gated_fwd(p["x"], p["g"], p["r"], p["A"], p["z"], h0=p["h0"], ckpt=ck)
        return {"y": y, "last": last, **selscan.gated_bwd(p["x"], p["g"], p["r"], p["A"], p["z"], dy=p["dy"],
                                                          h0=p["h0"], dlast_state=p["dlast"], ckpt=ck, want_dh0=True)}

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
        new = make(B, L, D, kind, torch.bfloat16, seed=13 + turn, z=True, h0=True, grads=True)
        for k in ("x", "g", "r", "z", "dy", "h0"):
            if p[k] is not None:
                p[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in out.items()}
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want), turn


def test_token_loop_in_a_graph():
    case("token loop in a graph")
    B, D = 3, 200
    p = make(B, 1, D, "decay", torch.bfloat16, seed=20, z=True, h0=True, one=True)
    state, eager = p["h0"].clone(), p["h0"].clone()
    selscan.gated_step(state.clone(), p["x"], p["g"], p["r"], p["A"], p["z"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = selscan.gated_step(state, p["x"], p["g"], p["r"], p["A"], p["z"])
    for turn in range(5):
        new = make(B, 1, D, "decay", torch.bfloat16, seed=21 + turn, z=True, one=True)
        for k in ("x", "g", "r", "z"):
            p[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        want = selscan.gated_step(eager, p["x"], p["g"], p["r"], p["A"], p["z"])
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(state, eager)


CHAINED = [
    # long and few channels: tiles in a chain (batch, tokens, channels)
    (1, 2048, 64),
    (1, 2049, 2),
    (2, 2200, 70),
    (1, 4097, 33),
    (3, 2311, 130),
    (1, 6000, 1),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", CHAINED)
def test_chained_tiles(shape, dtype, kind):
    """Against the definition; the gradients from the chain's checkpoints; whole, padded, from a state in place."""
    B, L, D = shape
    for z, h0 in ((False, False), (True, True)):
        lengths = [L - 700 * b for b in range(B)] if h0 else None
        what = f"chain {shape} {dtype} {kind} z={z} h0={h0}"
        case(what)
        p = make(B, L, D, kind, DT[dtype], seed=30, z=z, h0=h0, lengths=lengths, grads=True)
        q = np_of(p)
        y, last, c = forward(p, ckpt=True)
        check_fwd(y, last, q, what, c)
        check_bwd(backward(p, c), q, what)
        if h0:
            state = p["h0"].clone()
            y2, _ = selscan.gated_fwd(p["x"], p["g"], p["r"], p["A"], p["z"], h0=state, lengths=p["lengths"],
                                      last_state=state)
            torch.cuda.synchronize()
            assert torch.equal(y, y2) and torch.equal(last, state)


def test_chain_is_deterministic():
    """Over many calls, from workspaces of any contents, beside another call on another stream, in a graph."""
    case("chain, determinism")
    p = make(1, 9000, 200, "decay", torch.float32, seed=31, z=True, h0=True)
    q = make(1, 12000, 64, "mix", torch.bfloat16, seed=32)
    y, last, c = forward(p, ckpt=True)
    yq, lastq, _ = forward(q)
    need = selscan.gated_workspace_size(1, 9000, 200, torch.float32)
    ws, ws2 = (torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    for turn in range(12):
        ws.fill_(turn * 23 % 256)
        y2, last2, c2 = forward(p, ckpt=True, workspace=ws)
        assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(c, c2), turn
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a = selscan.gated_fwd(q["x"], q["g"])
        b = selscan.gated_fwd(p["x"], p["g"], p["r"], p["A"], p["z"], h0=p["h0"], workspace=ws2)
        torch.cuda.synchronize()
        assert torch.equal(a[0], yq) and torch.equal(a[1], lastq)
        assert torch.equal(b[0], y) and torch.equal(b[1], last)
    graphs = []
    for _ in range(2):  # two graphs that share a workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = selscan.gated_fwd(p["x"], p["g"], p["r"], p["A"], p["z"], h0=p["h0"], workspace=ws)
        graphs.append((g, out))
    for turn in range(3):
        for g, out in graphs:
            out[0].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], y) and torch.equal(out[1], last)
        p["x"].mul_(1.0)  # (the program's own work between the replays)


def test_chain_not_finite():
    case("chain, not finite")
    for kind in KINDS:
        p = make(1, 4000, 70, kind, torch.float32, seed=33)
        clean, _, _ = forward(p)
        p["x"][0, 1303, 17] = float("nan")
        p["g"][0, 2900, 68] = float("nan")
        y, last, _ = forward(p)
        same = torch.ones_like(y, dtype=torch.bool)
        same[0, 1303:, 17] = same[0, 2900:, 68] = False
        assert torch.equal(y[same], clean[same]) and torch.isnan(y[0, 1303:, 17]).all() and torch.isnan(last[0, 68])
        if kind == "decay":
            p["r"][0, :] = float("-inf")  # nothing is forgotten, nothing added
            p["x"].zero_()
            p["g"].zero_()
            y, last = selscan.gated_fwd(p["x"], p["g"], p["r"], p["A"], h0=torch.full((1, 70), 3.0, device="cuda"))
            torch.cuda.synchronize()
            assert (y == 3).all() and (last == 3).all()
