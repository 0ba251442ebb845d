"""The gated recurrence, the norms around a block and rotary positions past 2^31 and 2^32 values of a tensor: what
stands at the end of it against the definition, or against a call on that part alone. pytest -m gpu."""
import numpy as np
import pytest
import torch

from blocks_util import bounds, close, np_of
from oracle import blocks as ref
from selective_state_space_48_amd import selscan

pytestmark = pytest.mark.gpu


def case(msg):
    print(f"[case] {msg}", flush=True)


def fill(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in t.view(-1).chunk(16):
        part.normal_(generator=g)
    return t


@pytest.mark.parametrize("shape", [(1100, 1000, 4096), (1, 1 << 20, 2050), (1, 1 << 21, 2049)])
def test_gated_past_2_32_values(shape):
    """A walk a workgroup, chained tiles, and odd channels; the last entry's last channels, forward and backward."""
    B, L, D = shape
    case(f"gated {shape}")
    x, g = fill(shape, 1), fill(shape, 2)
    assert x.numel() > 1 << 31
    y, last = selscan.gated_fwd(x, g)
    chans = [0, D // 2, D - 2, D - 1]
    n = min(L, 3000)  # a state of some 2 tokens' memory: tokens further back reach nothing
    cut = lambda t: t[B - 1:, L - n:, chans].contiguous()  # noqa: E731
    q = np_of(dict(x=cut(x), g=cut(g), r=None, A=None, z=None, h0=None, lengths=None, dy=cut(g), dlast=None))
    k = bounds(q)
    wy, wl, _ = ref.gated(q["x"], q["g"])
    tail = slice(n // 2, n)
    close(cut(y)[:, tail].contiguous(), wy[:, tail], k["Ea"][:, tail], "y")
    close(last[B - 1:, chans].contiguous(), wl, k["E"], "last_state")
    del y
    r = selscan.gated_bwd(x, g, dy=g, want_dh0=True)
    torch.cuda.synchronize()
    want = ref.gated_bwd(q["x"], q["g"], q["dy"])
    # gradients come from tokens behind, of which the cut has them all; terms below 2^4, each within 100 roundings
    for name in ("dx", "dg"):
        close(cut(r[name])[:, tail].contiguous(), want[name][:, tail], 100 * 2.0 ** -24 * 16, name)


def test_addnorm_and_rotary_past_2_32_values():
    """Rows and tokens by themselves: the last ones are what a call on them alone gives."""
    R, C = 1_100_000, 4096
    case(f"addnorm {(R, C)}")
    x, res = fill((R, C), 3), fill((R, C), 4)
    w = torch.rand(C, device="cuda") + 0.5
    kw = dict(post="rms", post_weight=w, pre_weight=w)
    y, s, st = selscan.addnorm(x, res, **kw)
    tail = slice(R - 300, R)
    part = [t[tail].clone() for t in (x, res)]
    y2, s2, st2 = selscan.addnorm(*part, **kw)
    assert torch.equal(y[tail], y2) and torch.equal(s[tail], s2) and torch.equal(st[tail], st2)
    r = selscan.addnorm_bwd(x, s, dy=y, stats=st, **kw)
    r2 = selscan.addnorm_bwd(part[0], s2, dy=y2, stats=st2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(r["dx"][tail], r2["dx"]) and torch.equal(r["dres"][tail], r2["dres"])
    # a column's sum over all rows: y is pre's value times w, so sum y xh = w sum xh^2 up to y's rounding (2^-9 a term)
    xh2 = torch.zeros(C, dtype=torch.float64, device="cuda")
    for a in range(0, R, 100_000):
        xh2 += (s[a:a + 100_000].double() * st[a:a + 100_000, 3:4].double()).square().sum(0)
    want = (w.double() * xh2).cpu().numpy()
    # y and the stored sum are each rounded to bfloat16, by at most 2^-8 of the value (2^-8 / sqrt(3) root mean square,
    # sqrt(2) times that for both); over R normal terms the squares' sum is off by sqrt(3 / R) of that: 5.3e-6. The
    # largest of 4096 columns is below 5.7 of these, 2^-15.
    close(r["dpre_weight"], want, want * 2.0 ** -15, "dpre_weight over a million rows")
    case("rotary")
    q = x.view(1, R, 32, 128)
    inv = selscan.rotary_frequencies(128, device="cuda")
    qo, _ = selscan.rotary(q, None, inv, layout="interleaved")
    part, _ = selscan.rotary(q[:, tail].clone(), None, inv, layout="interleaved", offset=R - 300)
    torch.cuda.synchronize()
    assert torch.equal(qo[:, tail], part)
