"""The types of the norms' gradients where few tensors are given to say them."""
import pytest
import torch

from selective_state_space_48_amd import selscan as S

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rn(*s, dtype=F32, seed=0):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("C", [5, 96, 5000])
@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (BF, F32)])
def test_gradients_of_a_plain_sum_have_the_inputs_types(types, C):
    """res_out = 2 res + 0.5 x without norms: dx and dres come from dres_out alone, each rounded once to its type."""
    dt, rt = types
    print(f"[case] a plain sum, {dt} {rt} {C}", flush=True)
    ds, gate = rn(12, C, dtype=rt), rn(3, C, seed=1)
    for g in (None, gate):
        kw = dict(dy=None, dres_out=ds, stats=None, pre="none", scale=0.5, res_scale=2.0, gate=g, want_dparams=False)
        r = S.addnorm_bwd(None, None, **kw, dtype=dt)
        with_x = S.addnorm_bwd(rn(12, C, dtype=dt, seed=2), None, **kw)
        torch.cuda.synchronize()
        assert r["dx"].dtype == dt and r["dres"].dtype == rt
        du = 0.5 * ds.double() * (1.0 if g is None else g.double().repeat_interleave(4, 0))
        # products of one or two factors in fp32 (a half is exact), then half a step of the type
        room = du.abs() * (2.0 ** -24 + torch.finfo(dt).eps / 2 * (1 + 2.0 ** -24)) + 1e-37
        assert ((r["dx"].double() - du).abs() <= room).all()
        assert torch.equal(r["dres"].double(), 2 * ds.double())
        assert all(torch.equal(r[k], with_x[k]) for k in ("dx", "dres"))


def test_what_the_tensors_say_is_taken_without_a_name():
    print("[case] types as the tensors have them", flush=True)
    x, s = rn(6, 40, dtype=BF), rn(6, 40, seed=1)
    _, s, st = S.addnorm(x, s, pre="layer")
    r = S.addnorm_bwd(None, s, dy=x, stats=st, pre="layer")
    plain = S.addnorm_bwd(None, None, dy=None, dres_out=s, stats=None, pre="none")
    nothing = S.addnorm_bwd(x, None, dy=None, stats=None, pre="none", res_dtype=F32)
    torch.cuda.synchronize()
    assert r["dx"].dtype == BF and r["dres"].dtype == F32
    assert plain["dx"].dtype == F32 and torch.equal(plain["dx"], s)
    assert nothing["dx"].dtype == BF and nothing["dres"].dtype == F32 and (nothing["dres"] == 0).all()
