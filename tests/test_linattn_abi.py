"""Refusals of the linear-attention and group-norm calls, before any HIP call (CPU; fake pointers)."""
import ctypes
import random

import pytest
import torch

from selective_state_space_48_amd import selscan as S

BASE, STEP = 1 << 40, 1 << 32
lib = S.lib


def P(i):
    return ctypes.c_void_p(BASE + i * STEP)


def la(batch=2, seqlen=10, heads=4, kv_heads=2, dk=64, dv=32, dtype=S.BF16):
    return S.LinattnDims(batch, seqlen, heads, kv_heads, dk, dv, dtype)


def addr(p):
    return None if p is None else p.value


def fwd(d, ptrs=None, **o):
    p = ptrs or [P(i) for i in range(6)]
    opts = S.LinattnOpts(addr(o.get("h0")), addr(o.get("lengths")), o.get("scale", 0.0), o.get("segments", 0),
                         addr(o.get("ws")), o.get("ws_bytes", 0))
    return lib.selscan_linattn_fwd(*p, ctypes.byref(d) if d else None, ctypes.byref(opts), None)


def step(d, ptrs=None, scale=0.0):
    return lib.selscan_linattn_step(*(ptrs or [P(i) for i in range(6)]), ctypes.byref(d) if d else None, scale, None)


def bwd(d, ptrs=None, **o):
    p = ptrs or [P(i) for i in range(9)]
    opts = S.LinattnBwdOpts(addr(o.get("h0")), addr(o.get("lengths")), addr(o.get("dlast")), addr(o.get("dh0")),
                            o.get("scale", 0.0), o.get("segments", 0), addr(o.get("ws")), o.get("ws_bytes", 0))
    return lib.selscan_linattn_bwd(*p, ctypes.byref(d) if d else None, ctypes.byref(opts), None)


@pytest.mark.parametrize("call", [fwd, step, bwd])
def test_linattn_dims(call):
    assert call(None) == S.ERR_NULL
    for k in ("batch", "heads", "kv_heads", "dk", "dv"):
        assert call(la(**{k: -1})) == S.ERR_DIMS, k
    assert call(la(dtype=7)) == S.ERR_DTYPE
    for w in (0, 4, 12, 264, 260):
        assert call(la(dk=w)) == S.ERR_DSTATE and call(la(dv=w)) == S.ERR_DSTATE, w
    assert call(la(kv_heads=0)) == S.ERR_DIMS
    assert call(la(kv_heads=3)) == S.ERR_DIMS
    assert call(la(heads=2, kv_heads=4)) == S.ERR_DIMS
    assert call(la(heads=1 << 15, kv_heads=1)) == S.ERR_DIMS
    assert call(la(batch=1 << 62)) == S.ERR_DIMS
    assert call(la(batch=1 << 25)) == S.ERR_DIMS  # too many states for a grid
    for bad in (float("nan"), float("inf")):
        assert call(la(), scale=bad) == S.ERR_CONFIG
    if call is not step:
        assert call(la(seqlen=-1)) == S.ERR_DIMS
        assert call(la(seqlen=1 << 27)) == S.ERR_DIMS
        assert call(la(), segments=-1) == S.ERR_CONFIG
        assert call(la(), segments=65537) == S.ERR_CONFIG


@pytest.mark.parametrize("call,n,optional", [(fwd, 6, {5}), (step, 6, set()), (bwd, 9, {8})])
def test_linattn_pointers(call, n, optional):
    for i in range(n):
        ptrs = [P(k) for k in range(n)]
        if i not in optional:
            ptrs[i] = None
            assert call(la(), ptrs) == S.ERR_NULL, i
        ptrs[i] = ctypes.c_void_p(BASE + i * STEP + 8)
        assert call(la(), ptrs) == S.ERR_ALIGN, i


def test_linattn_alias():
    def at(i, j, n):  # argument i at argument j's place
        p = [P(k) for k in range(n)]
        p[i] = p[j]
        return p

    for i in (4, 5):
        for j in range(4):
            assert fwd(la(), at(i, j, 6)) == S.ERR_ALIAS
    assert fwd(la(), at(5, 4, 6)) == S.ERR_ALIAS
    assert fwd(la(), h0=P(4)) == S.ERR_ALIAS
    assert fwd(la(), h0=ctypes.c_void_p(P(5).value + 256)) == S.ERR_ALIAS  # half over last_state
    assert fwd(la(), lengths=P(4)) == S.ERR_ALIAS
    for i in (0, 5):
        for j in range(1, 5):
            assert step(la(), at(i, j, 6)) == S.ERR_ALIAS
    for i in range(5, 9):
        for j in range(i):
            assert bwd(la(), at(i, j, 9)) == S.ERR_ALIAS, (i, j)
    for j in range(9):
        assert bwd(la(), dh0=P(j)) == S.ERR_ALIAS, j
    assert bwd(la(), dh0=P(10), h0=P(10)) == S.ERR_ALIAS
    assert bwd(la(), dh0=P(10), dlast=P(10)) == S.ERR_ALIAS
    assert bwd(la(), lengths=P(6)) == S.ERR_ALIAS


def sizes(d, segments=0, slope=1):
    f, b = ctypes.c_uint64(1), ctypes.c_uint64(1)
    fo, bo = S.LinattnOpts(None, None, 0.0, segments, None, 0), S.LinattnBwdOpts(None, None, None, None, 0.0, segments)
    rc = (lib.selscan_linattn_fwd_workspace_size(ctypes.byref(d), ctypes.byref(fo), ctypes.byref(f)),
          lib.selscan_linattn_bwd_workspace_size(ctypes.byref(d), ctypes.byref(bo), slope, ctypes.byref(b)))
    return rc, f.value, b.value


def test_linattn_workspace():
    assert sizes(la())[0] == (S.OK, S.OK)
    assert sizes(la(seqlen=0)) == ((S.OK, S.OK), 0, 0)
    assert sizes(la(dk=3))[0] == (S.ERR_DSTATE, S.ERR_DSTATE)
    assert sizes(la(), segments=-1)[0] == (S.ERR_CONFIG, S.ERR_CONFIG)
    d = la()
    assert lib.selscan_linattn_fwd_workspace_size(ctypes.byref(d), None, None) == S.ERR_NULL
    assert lib.selscan_linattn_bwd_workspace_size(ctypes.byref(d), None, 0, None) == S.ERR_NULL
    # shared keys and values need room for the heads' own gradients
    assert sizes(la(), slope=0)[2] >= 2 * 10 * 4 * (64 + 32) * 4
    need = sizes(la())[2]
    assert bwd(la(), ws=P(20), ws_bytes=need - 1) == S.ERR_CONFIG
    assert bwd(la(), ws=ctypes.c_void_p(P(20).value + 16), ws_bytes=need) == S.ERR_CONFIG
    assert bwd(la(), ws=P(6), ws_bytes=need) == S.ERR_ALIAS


def test_linattn_automatic_runs():
    """Runs where heads leave CUs idle and the sequence is long enough (workspace: a state per run)."""
    def runs(**kw):
        d = la(kv_heads=4, dk=128, dv=128, **kw)
        return sizes(d)[1] // (d.batch * d.heads * 128 * 128 * 4)

    assert runs(batch=64, seqlen=100000) == 0      # 256 heads: one workgroup a CU already
    assert runs(batch=1, seqlen=300) == 0          # too short to pay for two launches
    # 4 heads: 64 runs make one round; of 100000 / 64 = 1562.5 tokens, rounded up to 1600: 62.5 of them
    assert runs(batch=1, seqlen=100000) == 63
    assert runs(batch=16, seqlen=100000) == 4
    assert runs(batch=1, seqlen=1024) == 8         # runs of 128 tokens
    assert sizes(la(batch=1 << 18, seqlen=3))[0] == (S.ERR_DIMS, S.ERR_DIMS)  # a grid of 2^32 threads
    assert sizes(la(batch=1 << 14, seqlen=10000), segments=100)[0] == (S.ERR_DIMS, S.ERR_DIMS)


def gn(batch=2, spatial=3, channels=32, groups=4, dtype=S.BF16, act=0, eps=1e-5):
    return S.GroupnormDims(batch, spatial, channels, groups, dtype, act, eps)


def gfwd(d, ptrs=None, ws=None, ws_bytes=0):
    """x, weight, bias, z, y, mean, rstd"""
    p = list(ptrs or [P(i) for i in range(7)])
    if ptrs is None and d is not None and d.act != 2:
        p[3] = None
    o = S.GroupnormOpts(addr(ws), ws_bytes)
    return lib.selscan_groupnorm(*p, ctypes.byref(d) if d else None, ctypes.byref(o), None)


def gbwd(d, ptrs=None, ws=None, ws_bytes=0):
    """x, weight, bias, z, dy, mean, rstd, dx, dweight, dbias, dz"""
    p = list(ptrs or [P(i) for i in range(11)])
    if ptrs is None and d is not None and d.act != 2:
        p[3] = p[10] = None
    o = S.GroupnormOpts(addr(ws), ws_bytes)
    return lib.selscan_groupnorm_bwd(*p, ctypes.byref(d) if d else None, ctypes.byref(o), None)


@pytest.mark.parametrize("call", [gfwd, gbwd])
def test_groupnorm_dims(call):
    assert call(None) == S.ERR_NULL
    for k in ("batch", "spatial", "channels", "groups"):
        assert call(gn(**{k: -1})) == S.ERR_DIMS, k
    assert call(gn(groups=0)) == S.ERR_DIMS
    assert call(gn(groups=5)) == S.ERR_DIMS
    assert call(gn(dtype=5)) == S.ERR_DTYPE
    assert call(gn(act=3)) == S.ERR_CONFIG
    assert call(gn(act=-1)) == S.ERR_CONFIG
    assert call(gn(batch=1 << 40)) == S.ERR_DIMS
    assert call(gn(channels=1 << 25)) == S.ERR_DIMS


def test_groupnorm_pointers():
    for bad in (-1.0, float("nan"), float("inf")):
        assert gfwd(gn(eps=bad)) == S.ERR_CONFIG
    for call, n, need, outs in ((gfwd, 7, (0, 3, 4, 5, 6), (4, 5, 6)), (gbwd, 11, (0, 3, 4, 5, 6, 7, 10), (7, 8, 9, 10))):
        full = [P(i) for i in range(n)]
        for i in range(n):
            p = list(full)
            if i in need:
                p[i] = None
                assert call(gn(act=2), p) == S.ERR_NULL, i
            p[i] = ctypes.c_void_p(BASE + i * STEP + 4)
            assert call(gn(act=2), p) == S.ERR_ALIGN, i
            for j in outs:
                if i != j:
                    p = list(full)
                    p[j] = p[i]
                    assert call(gn(act=2), p) == S.ERR_ALIAS, (i, j)
        assert call(gn(act=1), full) == S.ERR_NULL  # a gate that the activation does not use
    n = ctypes.c_uint64(0)
    d = gn()
    assert lib.selscan_groupnorm_workspace_size(ctypes.byref(d), 1, None) == S.ERR_NULL
    assert lib.selscan_groupnorm_workspace_size(ctypes.byref(d), 1, ctypes.byref(n)) == S.OK and n.value > 0
    assert gbwd(d, ws=P(20), ws_bytes=n.value - 1) == S.ERR_CONFIG
    assert gbwd(d, ws=ctypes.c_void_p(P(20).value + 8), ws_bytes=n.value) == S.ERR_CONFIG
    assert gbwd(d, ws=P(7), ws_bytes=n.value) == S.ERR_ALIAS


def gn_size(N, S, C, G, dtype=S.BF16, act=0):
    d, n = gn(N, S, C, G, dtype, act), [ctypes.c_uint64(0), ctypes.c_uint64(0)]
    return [lib.selscan_groupnorm_workspace_size(ctypes.byref(d), i, ctypes.byref(n[i])) for i in (0, 1)]


def test_groupnorm_sizes():
    """Every size that the header allows is taken, forwards and backwards: 2^32 threads of a workgroup for
    each entry and group are no limit where a workgroup takes many of them."""
    both = [S.OK, S.OK]
    for N in (131071, 131072, 1 << 20):
        assert gn_size(N, 2, 512, 512) == both, N   # small maps of many narrow groups
    assert gn_size(5_000_000, 1, 1025, 1, S.F32) == both  # rows wider than a workgroup's vectors
    assert gn_size(1 << 20, 3, 4097, 1) == both
    assert gn_size(1 << 16, 1 << 10, 128, 4) == both
    rng = random.Random(5)
    for _ in range(3000):
        log = lambda hi: int(2 ** rng.uniform(0, hi))  # noqa: E731
        G = log(10)
        C = G * log(14)
        rows = (1 << 33) // C
        N = max(1, min(log(33), rows - 1, (1 << 31) // G - 1))
        size = N, max(1, min(log(30), (rows - 1) // N)), C, G
        for dtype in (S.F32, S.BF16):
            for act in (0, 2):
                assert gn_size(*size, dtype, act) == both, (size, dtype, act)
    refused = [S.ERR_DIMS, S.ERR_DIMS]
    assert gn_size(1 << 30, 1, 8, 2) == refused
    assert gn_size(1, 1 << 31, 8, 2) == refused
    assert gn_size(1 << 24, 1 << 15, 64, 1) == refused  # 2^45 values


def test_binding_refusals():
    """Shapes, types, places and strides that the binding turns down itself."""
    z = torch.zeros
    q, k, v, g = z(2, 5, 4, 32), z(2, 5, 2, 32), z(2, 5, 2, 16), z(4)
    st = z(2, 4, 32, 16)
    ok = dict(q=q, k=k, v=v, log_decay=g)

    def f(**kw):
        a = dict(ok, **kw)
        return S.linattn_fwd(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("log_decay"), **a)

    for kw, e in ((dict(q=q[0]), ValueError), (dict(k=z(2, 5, 2, 31)), ValueError), (dict(v=z(2, 4, 2, 16)), ValueError),
                  (dict(k=k.bfloat16()), TypeError), (dict(q=q.half()), TypeError), (dict(log_decay=z(3)), ValueError),
                  (dict(log_decay=g.double()), TypeError), (dict(h0=z(2, 4, 16, 32)), ValueError),
                  (dict(lengths=z(2)), TypeError), (dict(lengths=z(3, dtype=torch.int32)), ValueError),
                  (dict(q=z(2, 5, 32, 4).transpose(2, 3)), ValueError), ({}, ValueError)):  # {}: not on a GPU
        with pytest.raises(e):
            f(**kw)
    with pytest.raises(ValueError):
        S.linattn_step(st, q, k, v, g)
    with pytest.raises(ValueError):
        S.linattn_bwd(q, k, v, g, dy=z(2, 5, 4, 32))
    x = z(6, 8)
    for kw, e in ((dict(act="relu"), ValueError), (dict(act="gate"), ValueError), (dict(z=x), ValueError),
                  (dict(weight=z(4)), ValueError), (dict(weight=z(8).bfloat16()), TypeError), ({}, ValueError)):
        with pytest.raises(e):
            S.groupnorm(x, 2, **kw)
    with pytest.raises(ValueError):
        S.groupnorm(z(2, 2, 2, 8), 2)
    with pytest.raises(ValueError):
        S.groupnorm_bwd(x, 2, dy=x, mean=z(6, 3), rstd=z(6, 2))


def test_binding_scale():
    """A scale that is 0 in fp32 is refused: the C calls would take it for the default."""
    for bad in (0, 0.0, -0.0, 1e-46, -1e-300):
        with pytest.raises(ValueError):
            S._scale(bad)
    assert S._scale(None) == 0 and S._scale(-0.5) == -0.5 and S._scale(1e-40) == 1e-40
