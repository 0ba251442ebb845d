"""Rotary positions on the GPU against the definition.

Tolerances: an angle's cosine and sine are off by at most 4 roundings U = 2^-24 of 1 (the turn's fraction formed in
64 bits: the product and the constant's rounding, 2^-51 of the turns, is below U up to 2^24 turns and 2^-20 at 2^31),
times the scale another rounding; the two products and their sum 3 more. The output's own rounding is half a step."""
import numpy as np
import pytest
import torch

from blocks_util import DT, U, close
from oracle import blocks as ref
from oracle import linattn as ref_la
from parity_util import to_np
from selective_state_space_48_amd import selscan

pytestmark = pytest.mark.gpu
LAYOUTS = ["half", "interleaved"]

SHAPES = [
    # batch, tokens, heads, kv heads, width, rot
    (1, 1, 1, 1, 2, 2),
    (2, 3, 2, 1, 6, 4),
    (1, 5, 3, 0, 10, 10),
    (2, 9, 4, 2, 64, 64),
    (1, 17, 5, 5, 64, 32),
    (3, 4, 8, 2, 128, 128),
    (1, 33, 2, 2, 80, 20),
    (2, 7, 3, 1, 96, 24),
    (1, 2, 40, 8, 128, 64),
    (1, 3, 1, 1, 256, 256),
    (1, 2, 2, 1, 1000, 514),
    (1, 2, 1, 2, 4096, 4096),
    (1, 300, 2, 1, 33, 16),
]


def case(msg):
    print(f"[case] {msg}", flush=True)


def rn(*s, dtype=torch.float32, seed=0):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def check(got, x, inv_freq, positions, layout, what, scale=1.0, inverse=False):
    want = ref.rotary(to_np(x), to_np(inv_freq), positions, layout, scale, inverse)
    rot = 2 * len(inv_freq)
    size = np.zeros(x.shape)
    size[..., :rot] = ref.rotary(np.abs(to_np(x)), np.zeros(rot // 2), positions * 0, layout, abs(scale))[..., :rot]
    other = np.abs(to_np(x))[..., :rot]
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    swapped = other.copy()
    swapped[..., lo], swapped[..., hi] = other[..., hi], other[..., lo]
    size[..., :rot] += abs(scale) * swapped
    turns = np.abs(positions).max() * float(inv_freq.max()) / 6.28 if positions.size else 0.0
    close(got, want, size * (8 * U + 6.3 * turns * 2.0 ** -51), what)
    if rot < x.shape[-1]:
        assert torch.equal(got[..., rot:], x[..., rot:]), what


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rotary(shape, dtype, layout):
    B, L, H, Hk, W, rot = shape
    case(f"rotary {shape} {dtype} {layout}")
    q, k = rn(B, L, H, W, dtype=DT[dtype], seed=1), rn(B, L, Hk, W, dtype=DT[dtype], seed=2) if Hk else None
    inv = selscan.rotary_frequencies(rot, device="cuda")
    rng = np.random.default_rng(3)
    for kw in (dict(), dict(inverse=True, scale=1.25), dict(offset=1000)):
        for given in (False, True):
            pos = rng.integers(0, 100000, (B, L)) if given else np.tile(np.arange(L), (B, 1))
            t = torch.tensor(pos, dtype=torch.int32, device="cuda") if given else None
            qo, ko = selscan.rotary(q, k, inv, positions=t, layout=layout, **kw)
            torch.cuda.synchronize()
            at = pos + kw.get("offset", 0)
            for got, x, n in ((qo, q, "q"), (ko, k, "k")):
                if x is not None:
                    check(got, x, inv, at, layout, f"{shape} {dtype} {layout} {kw} {n}", kw.get("scale", 1.0),
                          kw.get("inverse", False))


def test_far_and_negative_positions():
    case("far positions")
    x = rn(1, 8, 2, 32, seed=4)
    inv = selscan.rotary_frequencies(32, device="cuda")
    pos = np.array([[0, -1, -123456, 1 << 20, (1 << 24) + 1, 2 ** 30 + 7, 2 ** 31 - 1, -(2 ** 31)]])
    t = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for offset in (0, 2 ** 31 - 1, -(2 ** 31) + 1):
        q, _ = selscan.rotary(x, None, inv, positions=t, offset=offset)
        torch.cuda.synchronize()
        check(q, x, inv, pos + offset, "half", f"far, offset {offset}")


def test_in_place_and_back():
    case("in place and back")
    q, k = rn(2, 50, 4, 64, seed=5), rn(2, 50, 2, 64, seed=6)
    inv = selscan.rotary_frequencies(48, device="cuda")
    for layout in LAYOUTS:
        qo, ko = selscan.rotary(q, k, inv, layout=layout)
        q2, k2 = q.clone(), k.clone()
        r = selscan.rotary(q2, k2, inv, layout=layout, q_out=q2, k_out=k2)
        torch.cuda.synchronize()
        assert r[0] is q2 and torch.equal(q2, qo) and torch.equal(k2, ko)
        selscan.rotary(q2, k2, inv, layout=layout, inverse=True, q_out=q2, k_out=k2)
        torch.cuda.synchronize()
        close(q2, to_np(q), 32 * U * np.abs(to_np(q)).max(), f"back {layout}")


def test_tokens_one_by_one_and_empty():
    """A prompt's tokens one at a time, each at its position; no tokens, no heads."""
    case("tokens")
    q, k = rn(3, 6, 4, 64, dtype=torch.bfloat16, seed=7), rn(3, 6, 2, 64, dtype=torch.bfloat16, seed=8)
    inv = selscan.rotary_frequencies(64, device="cuda")
    want = selscan.rotary(q, k, inv)
    for t in range(6):
        got = selscan.rotary(q[:, t:t + 1].contiguous(), k[:, t:t + 1].contiguous(), inv, offset=t)
        assert torch.equal(got[0][:, 0], want[0][:, t]) and torch.equal(got[1][:, 0], want[1][:, t])
    for shape in ((0, 5, 2, 64), (2, 0, 2, 64), (2, 3, 0, 64)):
        e = torch.empty(shape, device="cuda")
        assert selscan.rotary(e, e, inv)[0].shape == shape
    torch.cuda.synchronize()


def test_gradient_is_the_turn_back():
    """<rotary(x), dy> = <x, rotary back(dy)>, and against differences of the definition."""
    case("gradient")
    x, dy = rn(2, 20, 3, 40, seed=9), rn(2, 20, 3, 40, seed=10)
    inv = selscan.rotary_frequencies(24, device="cuda")
    for layout in LAYOUTS:
        dx, _ = selscan.rotary(dy, None, inv, layout=layout, scale=1.5, inverse=True)
        torch.cuda.synchronize()
        pos = np.tile(np.arange(20), (2, 1))
        d = np.random.default_rng(11).standard_normal(x.shape)
        f = lambda v: (ref.rotary(v, to_np(inv), pos, layout, 1.5) * to_np(dy)).sum()  # noqa: E731
        diff = (f(to_np(x) + 1e-3 * d) - f(to_np(x) - 1e-3 * d)) / 2e-3
        # the scale turns the passed-on part too in neither direction
        got = (to_np(dx) * d).sum()
        assert abs(diff - got) <= 16 * U * 1.5 * 2 * np.abs(d).sum() * 5 + 1e-9


def test_graph():
    case("graph")
    q, k = rn(2, 9, 4, 64, dtype=torch.bfloat16, seed=12), rn(2, 9, 2, 64, dtype=torch.bfloat16, seed=13)
    inv = selscan.rotary_frequencies(64, device="cuda")
    pos = torch.zeros(2, 9, dtype=torch.int32, device="cuda")
    run = lambda: selscan.rotary(q, k, inv, positions=pos, layout="interleaved")  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for turn in range(4):
        q.copy_(rn(2, 9, 4, 64, dtype=torch.bfloat16, seed=20 + turn))
        pos.copy_(torch.randint(0, 9999, (2, 9)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_before_linear_attention():
    """What rotary positions are for: queries and keys of linear attention, whose products then depend on the tokens'
    distance alone: the layer's outputs are the same from any first position."""
    case("before linear attention")
    B, L, H, Hk, W = 1, 40, 4, 2, 64
    q, k, v = rn(B, L, H, W, seed=14), rn(B, L, Hk, W, seed=15), rn(B, L, Hk, W, seed=16)
    inv = selscan.rotary_frequencies(W, device="cuda")
    g = torch.log1p(-(2.0 ** -torch.arange(4, 8, device="cuda", dtype=torch.float32)))
    outs = []
    for offset in (0, 100003):
        qr, kr = selscan.rotary(q, k, inv, offset=offset)
        y, _ = selscan.linattn_fwd(qr, kr, v, g)
        torch.cuda.synchronize()
        outs.append(y)
        pos = np.tile(np.arange(L) + offset, (B, 1))
        rq, rk = (ref.rotary(to_np(t), to_np(inv), pos) for t in (q, k))
        want, _ = ref_la.linattn(rq, rk, to_np(v), to_np(g))
        size, _ = ref_la.linattn(np.abs(rq), np.abs(rk), np.abs(to_np(v)), to_np(g))
        # 8 roundings more of both factors, whose magnitudes a turn mixes (at most a factor of 2 each)
        close(y, want, size * ((L + 2 * W + 64) + 2 * 8 * 4) * U * 2, f"linear attention, offset {offset}")
