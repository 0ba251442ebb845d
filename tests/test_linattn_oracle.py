"""The 64-bit definitions that the GPU tests compare against: their gradients
against autograd through an independent quadratic form and against central
differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import linattn as ref


def _quadratic(q, k, v, g, scale, h0, n):
    """The layer as a masked product over all pairs of tokens, and its last state."""
    B, L, H, dk = q.shape
    per = H // k.shape[2]
    k, v = k.repeat_interleave(per, 2), v.repeat_interleave(per, 2)
    y, last = [], []
    for b in range(B):
        m = int(n[b])
        t = torch.arange(m, dtype=torch.float64)
        gap = t[:, None] - t[None, :]
        D = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp(min=0)), 0.0)
        s = torch.einsum("thk,shk->hts", q[b, :m], k[b, :m]) * D
        o = torch.einsum("hts,shv->thv", s, v[b, :m])
        o = o + torch.einsum("thk,hkv,ht->thv", q[b, :m], h0[b], torch.exp(g[:, None] * (t + 1)))
        w = torch.exp(g[:, None] * (m - 1 - t))
        last.append(torch.einsum("shk,shv,hs->hkv", k[b, :m], v[b, :m], w) + torch.exp(g * m)[:, None, None] * h0[b])
        y.append(torch.cat([scale * o, torch.zeros(L - m, H, v.shape[3], dtype=torch.float64)]))
    return torch.stack(y), torch.stack(last)


@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
def test_linattn_gradients(lengths):
    B, L, H, Hk, dk, dv, scale = 3, 9, 4, 2, 3, 5, 0.7
    gen = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    t = dict(q=rn(B, L, H, dk), k=rn(B, L, Hk, dk), v=rn(B, L, Hk, dv), g=-rn(H).abs(), h0=rn(B, H, dk, dv))
    dy, dlast = rn(B, L, H, dv), rn(B, H, dk, dv)
    for x in t.values():
        x.requires_grad_()
    n = [L] * B if lengths is None else lengths
    y, last = _quadratic(t["q"], t["k"], t["v"], t["g"], scale, t["h0"], n)
    a = {k: x.detach().numpy() for k, x in t.items()}
    ry, rs = ref.linattn(a["q"], a["k"], a["v"], a["g"], scale, a["h0"], lengths)
    np.testing.assert_allclose(ry, y.detach().numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(rs, last.detach().numpy(), rtol=1e-10, atol=1e-12)
    ((y * dy).sum() + (last * dlast).sum()).backward()
    r = ref.linattn_bwd(a["q"], a["k"], a["v"], a["g"], dy.numpy(), scale, a["h0"], lengths, dlast.numpy())
    for name, x in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dlog_decay", "g"), ("dh0", "h0")):
        np.testing.assert_allclose(r[name], t[x].grad.numpy(), rtol=1e-9, atol=1e-11, err_msg=name)

    def loss(**change):
        b = dict(a, **change)
        y, s = ref.linattn(b["q"], b["k"], b["v"], b["g"], scale, b["h0"], lengths)
        return (y * dy.numpy()).sum() + (s * dlast.numpy()).sum()

    rng = np.random.default_rng(2)
    for name, x in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dlog_decay", "g"), ("dh0", "h0")):
        d = rng.standard_normal(a[x].shape)
        e = 1e-6
        diff = (loss(**{x: a[x] + e * d}) - loss(**{x: a[x] - e * d})) / (2 * e)
        assert abs(diff - (r[name] * d).sum()) <= 1e-6 * (1 + abs(diff)), name


@pytest.mark.parametrize("act", ["none", "silu", "gate"])
def test_groupnorm_gradients(act):
    N, S, C, G = 3, 4, 12, 3
    rng = np.random.default_rng(3)
    a = dict(x=rng.standard_normal((N, S, C)), weight=rng.standard_normal(C), bias=rng.standard_normal(C),
             z=rng.standard_normal((N, S, C)) if act == "gate" else None)
    dy = rng.standard_normal((N, S, C))
    y, mean, rstd = ref.groupnorm(a["x"], G, a["weight"], a["bias"], a["z"], act)
    tx = torch.nn.functional.group_norm(torch.tensor(a["x"]).transpose(1, 2), G, torch.tensor(a["weight"]),
                                        torch.tensor(a["bias"])).transpose(1, 2)
    ty = tx if act == "none" else torch.nn.functional.silu(tx)
    if act == "gate":
        ty = tx * torch.nn.functional.silu(torch.tensor(a["z"]))
    np.testing.assert_allclose(y, ty.numpy(), rtol=1e-9, atol=1e-12)
    r = ref.groupnorm_bwd(a["x"], G, a["weight"], a["bias"], a["z"], act, dy, mean, rstd)

    def loss(**change):
        b = dict(a, **change)
        return (ref.groupnorm(b["x"], G, b["weight"], b["bias"], b["z"], act)[0] * dy).sum()

    for name in [n for n in a if a[n] is not None]:
        d = rng.standard_normal(a[name].shape)
        e = 1e-6
        diff = (loss(**{name: a[name] + e * d}) - loss(**{name: a[name] - e * d})) / (2 * e)
        assert abs(diff - (r["d" + name] * d).sum()) <= 1e-6 * (1 + abs(diff)), name
