"""The recurrence, the norms and the rotary positions on the GPU in calls that meet each other: outputs in place of
inputs, runs without tokens, two calls at once."""
import pytest
import torch

from blocks_util import DT, check_bwd, check_fwd, make, np_of
from selective_state_space_48_amd import selscan
from test_addnorm_gpu import check as check_norm, make as make_norm

pytestmark = pytest.mark.gpu


def case(msg):
    print(f"[case] {msg}", flush=True)


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("C", [100, 2560, 8192, 8200, 16384])
def test_norm_gradients_in_place(C, types):
    """dres in place of dres_out gives what dres beside it gives, where the sums over rows are a launch of their own
    too (they need dres_out)."""
    dt, rt = DT[types[0]], DT[types[1]]
    R, gates = 6, 3
    g = torch.Generator().manual_seed(1)
    rn = lambda *s, d=torch.float32: torch.randn(s, generator=g).to(d).cuda()  # noqa: E731
    x, res, dy, ds, gate = rn(R, C, d=dt), rn(R, C, d=rt), rn(R, C, d=dt), rn(R, C, d=rt), rn(gates, C)
    for post, pre in (("layer", "rms"), ("rms", "none")):
        w = dict(post_weight=rn(C), post_bias=rn(C), pre_weight=rn(C) if pre != "none" else None,
                 pre_bias=rn(C) if pre != "none" else None, gate=gate)
        kw = dict(pre=pre, post=post, scale=0.5, res_scale=0.25, **w)
        case(f"{C} {types} {post} {pre}")
        _, s, stats = selscan.addnorm(x, res, **kw)
        if pre == "none":
            args, bw = (x, None), dict(dy=None, stats=stats, **kw)
        else:
            args, bw = (x, s), dict(dy=dy, stats=stats, **kw)
        want = selscan.addnorm_bwd(*args, dres_out=ds, **bw)
        own = ds.clone()
        got = selscan.addnorm_bwd(*args, dres_out=own, dres=own, **bw)
        torch.cuda.synchronize()
        assert got["dres"].data_ptr() == own.data_ptr()
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("kind", ["mix", "decay"])
def test_runs_without_tokens(kind):
    """Runs that lie behind an entry's length leave its state as it was, whatever ran on the CUs before."""
    B, L, D = 64, 2100, 130
    big = make(B, 600, D, kind, torch.float32, seed=1, h0=True)
    big["h0"] = big["h0"] * 1e30
    lengths = [0, 1, 255, 256, 257, 700, 2100, 0] * (B // 8)
    p = make(B, L, D, kind, torch.float32, seed=2, h0=True, lengths=lengths, grads=True)
    q = np_of(p)
    args = (p["x"], p["g"], p["r"], p["A"])
    empty = [b for b in range(B) if lengths[b] == 0]
    for segments in (8, 3):
        case(f"runs without tokens {kind} {segments}")
        selscan.gated_fwd(big["x"], big["g"], big["r"], big["A"], h0=big["h0"])
        y, last = selscan.gated_fwd(*args, h0=p["h0"], lengths=p["lengths"], segments=segments)
        selscan.gated_fwd(big["x"], big["g"], big["r"], big["A"], h0=big["h0"])
        r = selscan.gated_bwd(*args, dy=p["dy"], h0=p["h0"], lengths=p["lengths"], dlast_state=p["dlast"],
                              segments=segments, want_dh0=True)
        torch.cuda.synchronize()
        assert torch.equal(last[empty], p["h0"][empty]) and torch.equal(r["dh0"][empty], p["dlast"][empty])
        check_fwd(y, last, q, f"runs without tokens {kind} {segments}")
        check_bwd(r, q, f"runs without tokens {kind} {segments}")


@pytest.mark.parametrize("kind", ["mix", "decay"])
def test_two_calls_at_once(kind):
    """Chained calls, calls in runs and their gradients on two streams at once give what they give alone."""
    p = make(1, 9000, 700, kind, torch.bfloat16, seed=3, z=True, h0=True, grads=True)
    args = (p["x"], p["g"], p["r"], p["A"], p["z"])

    def both(segments):
        y, last = selscan.gated_fwd(*args, h0=p["h0"], segments=segments)
        r = selscan.gated_bwd(*args, dy=p["dy"], h0=p["h0"], dlast_state=p["dlast"], segments=segments, want_dh0=True)
        return [y, last, *(r[k] for k in sorted(r))]

    case(f"two calls at once {kind}")
    want = {s: both(s) for s in (0, 4)}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for st, s in zip(streams, (0, 0)):
            with torch.cuda.stream(st):
                got.append((s, both(s)))
    for st, s in zip(streams, (0, 4)):
        with torch.cuda.stream(st):
            got.append((s, both(s)))
    torch.cuda.synchronize()
    for s, outs in got:
        for a, b in zip(outs, want[s]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("C", [3, 8, 9, 15, 16, 17, 520, 4095, 4096, 4103, 5120, 5121, 6144, 6145, 7001, 8191, 8193, 9001])
def test_norms_where_the_split_changes(C, types):
    """Rows of a vector and its neighbours, and where threads of a row or vectors of a thread change: with gates and
    biases, with weights alone, and without a gradient of either."""
    for gates, bias, weight, post, pre in ((3, True, True, "layer", "rms"), (0, False, True, "rms", "layer"),
                                           (0, True, True, "rms", "rms"), (3, False, False, "none", "layer")):
        p = make_norm(6, C, types, seed=C, post=post, pre=pre, gates=gates, bias=bias, weight=weight)
        check_norm(p, post, pre, f"{C} {types} gates={gates} bias={bias} {post} {pre}")


@pytest.mark.parametrize("C", [5, 100, 2049, 4100, 9001])
def test_norms_in_place_and_beside(C):
    """res_out in place of res, where a row's last vector also reads values of its neighbour: the same bits, and
    nothing past the tensors' ends is written."""
    g = torch.Generator().manual_seed(C)
    R = 700
    x, res = (torch.randn(R, C, generator=g).bfloat16().cuda() for _ in range(2))
    for post, pre in (("none", "none"), ("rms", "layer")):
        case(f"{C} {post} {pre}")
        y, s, stats = selscan.addnorm(x, res, pre=pre, post=post)
        room = torch.full((R * C + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        own = room[:R * C].view(R, C)
        own.copy_(res)
        y2, s2, stats2 = selscan.addnorm(x, own, pre=pre, post=post, res_out=own)
        torch.cuda.synchronize()
        assert s2.data_ptr() == own.data_ptr() and torch.equal(s, own) and torch.equal(stats, stats2)
        assert (room[R * C:] == 7.0).all() and (y is None or torch.equal(y, y2))
