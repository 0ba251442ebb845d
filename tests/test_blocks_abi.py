"""Refusals of the gated recurrence, of the norms around a block and of rotary positions, before any HIP call (CPU;
fake pointers), and what the binding itself turns down."""
import ctypes
import math

import pytest
import torch

from selective_state_space_48_amd import selscan as S

BASE, STEP = 1 << 40, 1 << 34
lib = S.lib


def P(i):
    return ctypes.c_void_p(BASE + i * STEP)


def addr(p):
    return None if p is None else p.value


def ref(d):
    return ctypes.byref(d) if d is not None else None


def ga(batch=2, seqlen=100, dim=64, dtype=S.BF16, kind=S.GATED_DECAY):
    return S.GatedDims(batch, seqlen, dim, dtype, kind)


def ptrs_of(given, n, d, drop):
    p = list(given or [P(i) for i in range(n)])
    if given is None and d is not None and d.kind == S.GATED_MIX:
        for i in drop:
            p[i] = None
    return p


def gfwd(d, ptrs=None, **o):
    """x, g, r, A, z, y, last_state"""
    opts = S.GatedOpts(addr(o.get("h0")), addr(o.get("lengths")), addr(o.get("ckpt")), o.get("segments", 0),
                       addr(o.get("ws")), o.get("ws_bytes", 0))
    return lib.selscan_gated_fwd(*ptrs_of(ptrs, 7, d, (2, 3)), ref(d), ctypes.byref(opts), None)


def gstep(d, ptrs=None):
    """state, x, g, r, A, z, y"""
    return lib.selscan_gated_step(*ptrs_of(ptrs, 7, d, (3, 4)), ref(d), None)


def gbwd(d, ptrs=None, **o):
    """x, g, r, A, z, dy, dx, dg, dr, dA, dz"""
    opts = S.GatedBwdOpts(addr(o.get("h0")), addr(o.get("lengths")), addr(o.get("dlast")), addr(o.get("dh0")),
                          addr(o.get("ckpt")), o.get("segments", 0), addr(o.get("ws")), o.get("ws_bytes", 0))
    return lib.selscan_gated_bwd(*ptrs_of(ptrs, 11, d, (2, 3, 8, 9)), ref(d), ctypes.byref(opts), None)


@pytest.mark.parametrize("call", [gfwd, gstep, gbwd])
def test_gated_dims(call):
    assert call(None) == S.ERR_NULL
    for k in ("batch", "dim"):
        assert call(ga(**{k: -1})) == S.ERR_DIMS, k
    assert call(ga(dtype=7)) == S.ERR_DTYPE
    for kind in (-1, 2):
        assert call(ga(kind=kind)) == S.ERR_CONFIG
    assert call(ga(dim=(1 << 24) + 1)) == S.ERR_DIMS
    assert call(ga(batch=1 << 62)) == S.ERR_DIMS
    assert call(ga(batch=(1 << 22) // 8 + 1)) == S.ERR_DIMS
    if call is not gstep:
        assert call(ga(seqlen=-1)) == S.ERR_DIMS
        assert call(ga(seqlen=1 << 27)) == S.ERR_DIMS
        assert call(ga(), segments=-1) == S.ERR_CONFIG
        assert call(ga(), segments=65537) == S.ERR_CONFIG


@pytest.mark.parametrize("call,n,optional,decay_only", [
    (gfwd, 7, {4, 6}, (2, 3)), (gstep, 7, {5}, (3, 4)), (gbwd, 11, {9}, (2, 3, 8, 9))])
def test_gated_pointers(call, n, optional, decay_only):
    for i in range(n):
        ptrs = [P(k) for k in range(n)]
        if i not in optional:
            ptrs[i] = None
            assert call(ga(), ptrs) == S.ERR_NULL, i
        ptrs[i] = ctypes.c_void_p(BASE + i * STEP + 8)
        assert call(ga(), ptrs) == S.ERR_ALIGN, i
    for i in decay_only:  # what the other kind has no use for
        ptrs = [P(k) if k not in decay_only or k == i else None for k in range(n)]
        assert call(ga(kind=S.GATED_MIX), ptrs) == S.ERR_CONFIG, i


def test_gated_alias():
    def at(i, j, n):  # argument i at argument j's place
        p = [P(k) for k in range(n)]
        p[i] = p[j]
        return p

    for i in (5, 6):
        for j in range(5):
            assert gfwd(ga(), at(i, j, 7)) == S.ERR_ALIAS, (i, j)
    assert gfwd(ga(), at(6, 5, 7)) == S.ERR_ALIAS
    for name in ("h0", "lengths", "ckpt"):
        assert gfwd(ga(), **{name: P(5)}) == S.ERR_ALIAS, name
    assert gfwd(ga(), ckpt=P(0)) == S.ERR_ALIAS
    assert gfwd(ga(), ckpt=P(10), h0=P(10)) == S.ERR_ALIAS
    assert gfwd(ga(), h0=ctypes.c_void_p(P(6).value + 256)) == S.ERR_ALIAS  # half over last_state
    assert gfwd(ga(), lengths=P(6)) == S.ERR_ALIAS
    for i in (0, 6):
        for j in range(7):
            if i != j:
                assert gstep(ga(), at(i, j, 7)) == S.ERR_ALIAS, (i, j)
    for i in range(6, 11):
        for j in range(i):
            assert gbwd(ga(), at(i, j, 11)) == S.ERR_ALIAS, (i, j)
    for j in range(11):
        assert gbwd(ga(), dh0=P(j)) == S.ERR_ALIAS, j
    for name in ("h0", "dlast", "ckpt", "lengths"):
        assert gbwd(ga(), **{name: P(6)}) == S.ERR_ALIAS, name
        assert gbwd(ga(), dh0=P(12), **{name: P(12)}) == S.ERR_ALIAS, name


def gated_size(d, backward, segments=0, ckpt=False):
    n = ctypes.c_uint64(0)
    if backward:
        o = S.GatedBwdOpts(ckpt=16 if ckpt else None, segments=segments)
        return lib.selscan_gated_bwd_workspace_size(ref(d), ctypes.byref(o), ctypes.byref(n)), n.value
    return lib.selscan_gated_fwd_workspace_size(ref(d), ctypes.byref(S.GatedOpts(segments=segments)),
                                                ctypes.byref(n)), n.value


def test_gated_workspace():
    for backward in (False, True):
        assert gated_size(ga(seqlen=0), backward) == (S.OK, 0)
        assert gated_size(ga(dim=0), backward) == (S.OK, 0)
        assert gated_size(ga(kind=5), backward)[0] == S.ERR_CONFIG
        assert gated_size(ga(), backward, segments=-1)[0] == S.ERR_CONFIG
    d = ga()
    assert lib.selscan_gated_fwd_workspace_size(ref(d), None, None) == S.ERR_NULL
    assert lib.selscan_gated_bwd_workspace_size(ref(d), None, None) == S.ERR_NULL
    need = gated_size(d, True)[1]
    # states are kept where no checkpoints are given
    assert need >= gated_size(d, True, ckpt=True)[1] + 2 * 2 * 64 * 4
    assert gbwd(d, ws=P(20), ws_bytes=need - 1) == S.ERR_CONFIG
    assert gbwd(d, ws=ctypes.c_void_p(P(20).value + 16), ws_bytes=need) == S.ERR_CONFIG
    assert gbwd(d, ws=P(6), ws_bytes=need) == S.ERR_ALIAS
    assert gbwd(d, ws=P(0), ws_bytes=need) == S.ERR_ALIAS


def test_gated_automatic_splits():
    """Chained tiles where channels are few and tokens many (workspace: two words a tile and channel, one a link of 8
    tiles); runs of tokens backward (a stretch and a state each)."""
    def forward(**kw):
        return gated_size(ga(**kw), False)[1]

    assert forward(batch=1, seqlen=1024, dim=64) == 0      # too short to pay for it
    assert forward(batch=8, seqlen=4096, dim=4096) == 0    # two workgroups for every CU
    assert forward(batch=2, seqlen=4096, dim=4096) == 0    # narrow ones fill the CUs
    tiles, rows = 32, 2 * 64
    assert 0 <= forward(seqlen=4096) - (2 * tiles + 4) * rows * 8 - 256 - rows * 4 < 1024
    assert forward(seqlen=4097) > forward(seqlen=4096)

    def runs(**kw):  # one run needs no workspace with checkpoints and no dA
        d = ga(kind=S.GATED_MIX, **kw)
        return gated_size(d, True, ckpt=True)[1] / (d.batch * d.dim * 24)

    assert runs(batch=8, seqlen=4096, dim=4096) == 0
    assert runs(batch=1, seqlen=512, dim=64) == 0
    assert runs(batch=1, seqlen=16384, dim=512) == 32
    assert runs(batch=8, seqlen=2048, dim=64) == 16
    assert gated_size(ga(batch=1 << 18, dim=8), False, segments=65536)[0] == S.OK      # 100 tokens: one tile
    assert gated_size(ga(batch=1 << 18, dim=8, seqlen=1 << 14), False, segments=64)[0] == S.ERR_DIMS


def an(rows=12, channels=64, gate_rows=3, dtype=S.BF16, res_dtype=S.F32, post=1, pre=2, eps=1e-5, scale=1.0,
       res_scale=1.0):
    return S.AddnormDims(rows, channels, gate_rows, dtype, res_dtype, post, pre, eps, scale, res_scale)


def anorm(d, ptrs=None, params=None, ws=None):
    """x, res, res_out, y, stats; post_weight, post_bias, pre_weight, pre_bias, gate"""
    p = list(ptrs or [P(i) for i in range(5)])
    o = S.AddnormOpts(*(addr(t) for t in (params or [P(i) for i in range(5, 10)])))
    return lib.selscan_addnorm(*p, ref(d), ctypes.byref(o), None)


def anorm_bwd(d, ptrs=None, params=None, grads=None, ws=None, ws_bytes=1 << 40):
    """x, sum, stats, dy, dres_out, dx, dres; params; gradients of params"""
    p = list(ptrs or [P(i) for i in range(7)])
    o = S.AddnormOpts(*(addr(t) for t in (params or [P(i) for i in range(7, 12)])), addr(ws), ws_bytes if ws else 0)
    g = S.AddnormGrads(*(addr(t) for t in (grads or [P(i) for i in range(12, 17)])))
    return lib.selscan_addnorm_bwd(*p, ctypes.byref(g), ref(d), ctypes.byref(o), None)


@pytest.mark.parametrize("call", [anorm, anorm_bwd])
def test_addnorm_dims(call):
    assert call(None) == S.ERR_NULL
    for k in ("rows", "channels"):
        assert call(an(**{k: -1})) == S.ERR_DIMS, k
    assert call(an(rows=1 << 31, gate_rows=1)) == S.ERR_DIMS
    assert call(an(channels=65537)) == S.ERR_DIMS
    for gates in (0, -1, 5, 13):
        assert call(an(gate_rows=gates)) == S.ERR_DIMS, gates
    assert call(an(dtype=3)) == S.ERR_DTYPE
    assert call(an(res_dtype=3)) == S.ERR_DTYPE
    assert call(an(dtype=S.F32, res_dtype=S.BF16)) == S.ERR_DTYPE
    for k in ("post", "pre"):
        for v in (-1, 3):
            assert call(an(**{k: v})) == S.ERR_CONFIG, (k, v)
    for k in ("scale", "res_scale"):
        for v in (float("nan"), float("inf")):
            assert call(an(**{k: v})) == S.ERR_CONFIG, (k, v)
    if call is anorm:
        for v in (float("nan"), float("inf"), -1.0):
            assert call(an(eps=v)) == S.ERR_CONFIG, v


def test_addnorm_params_of_no_norm():
    none = [None] * 5
    for at, kw in ((0, dict(post=0)), (1, dict(post=0)), (2, dict(pre=0)), (3, dict(pre=0))):
        params = list(none)
        params[at] = P(20)
        ptrs = [P(i) for i in range(5)]
        if "pre" in kw:
            ptrs[3] = None
        assert anorm(an(**kw), ptrs, params) == S.ERR_CONFIG
        bp = [P(i) for i in range(7)]
        if "pre" in kw:
            bp[1] = bp[3] = None
        assert anorm_bwd(an(**kw), bp, params, none) == S.ERR_CONFIG
        assert anorm_bwd(an(**kw), bp, none, params) == S.ERR_CONFIG
    assert anorm(an(pre=0), None, none) == S.ERR_CONFIG            # a y that is not formed
    assert anorm_bwd(an(pre=0), None, none, none) == S.ERR_CONFIG  # a sum and dy that are not read
    assert anorm_bwd(an(), None, none, [None] * 4 + [P(20)]) == S.ERR_CONFIG  # a gate's gradient without a gate


def test_addnorm_pointers():
    none = [None] * 5
    for i, need in ((0, True), (1, False), (2, False), (3, True), (4, False)):
        p = [P(k) for k in range(5)]
        if need:
            p[i] = None
            assert anorm(an(), p) == S.ERR_NULL, i
        p[i] = ctypes.c_void_p(BASE + i * STEP + 4)
        assert anorm(an(), p) == S.ERR_ALIGN, i
    assert anorm(an(pre=0), [P(0), P(1), None, None, P(4)], none) == S.ERR_NULL  # nothing to write
    for i, need in ((0, True), (1, True), (2, True), (3, True), (4, False), (5, False), (6, False)):
        p = [P(k) for k in range(7)]
        if need:
            p[i] = None
            assert anorm_bwd(an(), p) == S.ERR_NULL, i
        p[i] = ctypes.c_void_p(BASE + i * STEP + 4)
        assert anorm_bwd(an(), p) == S.ERR_ALIGN, i
    assert anorm_bwd(an(), [P(k) for k in range(5)] + [None, None]) == S.ERR_NULL
    assert anorm_bwd(an(post=0), [None] + [P(k) for k in range(1, 7)], [None] * 4 + [P(20)],
                     [None] * 4 + [P(21)]) == S.ERR_NULL  # the gate's gradient reads x
    for k in range(5):
        params = [P(i) for i in range(20, 25)]
        params[k] = ctypes.c_void_p(P(20).value + 4)
        assert anorm(an(), None, params) == S.ERR_ALIGN
        assert anorm_bwd(an(), None, params) == S.ERR_ALIGN
        assert anorm_bwd(an(), None, None, params) == S.ERR_ALIGN


def test_addnorm_alias():
    for out in (2, 3, 4):
        for j in range(10):
            p, q = [P(k) for k in range(5)], [P(k) for k in range(5, 10)]
            if j == out or (out, j) == (2, 1):
                continue
            p[out] = P(j)
            assert anorm(an(), p, q) == S.ERR_ALIAS, (out, j)
    half = [P(k) for k in range(5)]
    half[2] = ctypes.c_void_p(P(1).value + 256)
    assert anorm(an(), half) == S.ERR_ALIAS  # half over res
    for out in (5, 6, 12, 13, 14, 15, 16):
        for j in range(17):
            allp = [P(k) for k in range(17)]
            if j == out or (out, j) == (6, 4):
                continue
            allp[out] = P(j)
            assert anorm_bwd(an(), allp[:7], allp[7:12], allp[12:]) == S.ERR_ALIAS, (out, j)
    half = [P(k) for k in range(7)]
    half[6] = ctypes.c_void_p(P(4).value + 256)
    assert anorm_bwd(an(), half) == S.ERR_ALIAS


def test_addnorm_workspace():
    n = ctypes.c_uint64(0)
    d, o, g = an(), S.AddnormOpts(gate=P(1).value), S.AddnormGrads(*(addr(P(i)) for i in range(5)))
    size = lib.selscan_addnorm_bwd_workspace_size
    assert size(ref(d), ctypes.byref(o), ctypes.byref(g), None) == S.ERR_NULL
    assert size(ref(an(pre=7)), ctypes.byref(o), ctypes.byref(g), ctypes.byref(n)) == S.ERR_CONFIG
    assert size(ref(d), None, None, ctypes.byref(n)) == S.OK and n.value == 0  # no sums over rows
    assert size(ref(an(rows=0)), ctypes.byref(o), ctypes.byref(g), ctypes.byref(n)) == S.OK and n.value == 0
    assert size(ref(d), ctypes.byref(o), ctypes.byref(g), ctypes.byref(n)) == S.OK and n.value > 0
    assert anorm_bwd(d, ws=P(20), ws_bytes=n.value - 1) == S.ERR_CONFIG
    assert anorm_bwd(d, ws=ctypes.c_void_p(P(20).value + 8)) == S.ERR_CONFIG
    for j in (0, 5, 12):
        assert anorm_bwd(d, ws=P(j)) == S.ERR_ALIAS, j


def ro(batch=2, seqlen=10, heads=4, kv_heads=2, width=64, rot=32, offset=0, dtype=S.BF16, layout=0, inverse=0, scale=0.0):
    return S.RotaryDims(batch, seqlen, heads, kv_heads, width, rot, offset, dtype, layout, inverse, scale)


def rotary(d, ptrs=None):
    """q, k, inv_freq, positions, q_out, k_out"""
    return lib.selscan_rotary(*(ptrs or [P(i) for i in range(6)]), ref(d), None)


def test_rotary_refusals():
    assert rotary(None) == S.ERR_NULL
    for k in ("batch", "seqlen", "heads", "kv_heads"):
        assert rotary(ro(**{k: -1})) == S.ERR_DIMS, k
    assert rotary(ro(seqlen=1 << 27)) == S.ERR_DIMS
    assert rotary(ro(batch=1 << 40)) == S.ERR_DIMS
    assert rotary(ro(heads=1 << 62, kv_heads=1 << 62)) == S.ERR_DIMS
    assert rotary(ro(heads=(1 << 16) - 1, kv_heads=2)) == S.ERR_DIMS
    assert rotary(ro(dtype=9)) == S.ERR_DTYPE
    for rot, width in ((0, 64), (-2, 64), (3, 64), (66, 64), (64, 4097)):
        assert rotary(ro(rot=rot, width=width)) == S.ERR_DSTATE, (rot, width)
    for off in (1 << 31, -(1 << 31)):
        assert rotary(ro(offset=off)) == S.ERR_DIMS
    for v in (-1, 2):
        assert rotary(ro(layout=v)) == S.ERR_CONFIG
    for v in (float("nan"), float("inf")):
        assert rotary(ro(scale=v)) == S.ERR_CONFIG
    for i in range(6):
        p = [P(k) for k in range(6)]
        if i != 3:
            p[i] = None
            assert rotary(ro(), p) == S.ERR_NULL, i
        p[i] = ctypes.c_void_p(BASE + i * STEP + 4)
        assert rotary(ro(), p) == S.ERR_ALIGN, i
    for out in (4, 5):
        for j in range(6):
            if j == out or (out, j) in ((4, 0), (5, 1)):  # in place
                continue
            p = [P(k) for k in range(6)]
            p[out] = P(j)
            assert rotary(ro(), p) == S.ERR_ALIAS, (out, j)
        p = [P(k) for k in range(6)]
        p[out] = ctypes.c_void_p(P(out - 4).value + 128)
        assert rotary(ro(), p) == S.ERR_ALIAS, out


def test_binding_refusals():
    """Shapes, types, places and strides that the binding turns down itself."""
    z = torch.zeros
    x, A = z(2, 5, 8), z(8)
    for a, kw, e in (((x[0], x[0]), {}, ValueError), ((x, z(2, 5, 7)), {}, ValueError), ((x, x.half()), {}, TypeError),
                     ((x.half(), x.half()), {}, TypeError), ((x, x, x), {}, ValueError), ((x, x, None, A), {}, ValueError),
                     ((x, x, x, A.double()), {}, TypeError), ((x, x, x, z(7)), {}, ValueError),
                     ((x, x), dict(h0=z(2, 7)), ValueError), ((x, x), dict(lengths=z(2)), TypeError),
                     ((x, x), dict(ckpt=z(2, 2, 8)), ValueError), ((x.transpose(0, 1), x.transpose(0, 1)), {}, ValueError),
                     ((x, x), {}, ValueError)):  # the last: not on a GPU
        with pytest.raises(e):
            S.gated_fwd(*a, **kw)
    with pytest.raises(ValueError):
        S.gated_bwd(x, x, dy=z(2, 4, 8))
    with pytest.raises(ValueError):
        S.gated_step(z(2, 5, 8), x, x)
    with pytest.raises(TypeError):
        S.gated_step(z(2, 8).double(), z(2, 8), z(2, 8))
    x = z(6, 8)
    for a, kw, e in (((x, z(6, 7)), {}, ValueError), ((x, x.bfloat16()), dict(pre="rms"), S.SelscanError),
                     ((x,), dict(pre="batch"), ValueError), ((x,), dict(pre_weight=z(7)), ValueError),
                     ((x,), dict(gate=z(8)), ValueError), ((x,), dict(gate=z(0, 8)), ValueError), ((x,), dict(gate=z(2, 7)), ValueError),
                     ((x.half(),), {}, TypeError), ((x.t(),), {}, ValueError), ((x,), {}, ValueError)):
        with pytest.raises((e, ValueError) if e is S.SelscanError else e):
            S.addnorm(*a, **kw)
    with pytest.raises(ValueError):
        S.addnorm_bwd(None, None, dy=None, stats=None)
    with pytest.raises(ValueError):
        S.addnorm_bwd(x, x, dy=x, stats=z(6, 3))
    q, f = z(2, 3, 4, 16), z(8)
    for a, kw, e in (((q[0], None, f), {}, ValueError), ((q, z(2, 3, 4, 8), f), {}, ValueError),
                     ((q, q.bfloat16(), f), {}, TypeError), ((q, None, f.double()), {}, TypeError),
                     ((q, None, f), dict(layout="pairs"), ValueError), ((q, None, f), dict(scale=0.0), ValueError),
                     ((q, None, f), dict(positions=z(2, 3)), TypeError), ((q, None, f), dict(k_out=q), ValueError),
                     ((q, None, z(2, 4)), {}, ValueError), ((q, None, f), {}, ValueError)):
        with pytest.raises(e):
            S.rotary(*a, **kw)


def test_rotary_frequencies():
    f = S.rotary_frequencies(64)
    assert f.dtype == torch.float32 and f[0] == 1 and abs(float(f[-1]) - 10000 ** (-62 / 64)) < 1e-10
    assert torch.equal(S.rotary_frequencies(64, scaling="linear", factor=4.0), f / 4)
    b = S.rotary_frequencies(64, scaling="base", factor=8.0)
    assert b[0] == 1 and abs(float(b[-1] / f[-1]) - 1 / 8) < 1e-6 and (b[1:] < f[1:]).all()
    p = S.rotary_frequencies(64, scaling="parts", factor=8.0, original=4096)
    turns = 4096 * f.double() / (2 * math.pi)
    assert torch.equal(p[turns > 64], f[turns > 64])
    assert torch.allclose(p[turns < 0.5], f[turns < 0.5] / 8, rtol=1e-6)
    assert (p <= f).all() and (p >= f / 8 * 0.999999).all()
    for kw in (dict(rot=7), dict(rot=0), dict(rot=8, base=1.0), dict(rot=8, factor=0), dict(rot=2, scaling="base"),
               dict(rot=8, scaling="parts"), dict(rot=8, scaling="cubic")):
        with pytest.raises(ValueError):
            S.rotary_frequencies(**kw)


@pytest.mark.parametrize("call", [gfwd, gstep, gbwd])
def test_gated_entries_without_channels(call):
    """The bound on entries holds without channels too, where no product of sizes says anything."""
    assert call(ga(batch=(1 << 22) + 1, dim=0)) == S.ERR_DIMS
    assert call(ga(batch=1 << 62, dim=0)) == S.ERR_DIMS


@pytest.mark.parametrize("call", [anorm, anorm_bwd])
def test_addnorm_gates_without_rows(call):
    """Any number of gate rows divides no rows; it is bounded as rows are."""
    for gates in (1 << 31, 1 << 62):
        assert call(an(rows=0, gate_rows=gates)) == S.ERR_DIMS


def test_gate_without_axes():
    x = torch.zeros(6, 8)
    for gate in (torch.zeros(()), torch.zeros(2, 3, 8)):
        with pytest.raises(ValueError):
            S.addnorm(x, gate=gate)
        with pytest.raises(ValueError):
            S.addnorm_bwd(x, x, dy=x, stats=torch.zeros(6, 4), gate=gate)
