"""The activations' derivatives far out in both tails, and the tail of gelu
relative to its own size, on the GPU against 64 bits."""
from __future__ import annotations

import pytest

from test_gpu_ffn import ACTS, U, _act_id, _f, igc, torch, ws  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
def test_slopes_of_extreme_sums(torch, igc, ws, act):  # noqa: F811
    """dbias of one row of ones is the slope itself.  Past |z| = 300 every derivative is 0 or 1 to the last bit of fp32."""
    big = [300.0, 1e4, 1e10, 1.5e19, 2e19, 1e20, 1e30, 3e38]
    z = torch.tensor([s * v for v in big for s in (1.0, -1.0)], device="cuda").bfloat16()
    N = z.numel()
    dY, db = torch.ones_like(z), torch.empty(N, device="cuda")
    kw = dict(Z=z, ldz=N, dbias=db, act=_act_id(igc, act), workspace=ws)
    igc.linear_backward(1, N, 8, dY, N, **kw)
    f, ref = (t.float() for t in _f(act, z.double()))
    assert bool(((ref == 0) | (ref == 1)).all())
    assert torch.equal(db, ref), (act, db, ref)
    # the gated block: dU = dH act(G) and dG = dH U act'(G)
    dbg, dbu = torch.empty_like(db), torch.empty_like(db)
    igc.glu_backward(1, N, 8, dY, N, z, N, dY, N, dbias_g=dbg, dbias_u=dbu, act=_act_id(igc, act), workspace=ws)
    assert torch.equal(dbg, ref) and torch.equal(dbu, f)


def test_tail_of_gelu_relative_to_its_size(torch, igc, ws):  # noqa: F811
    """fp32 outputs down to gelu(-12.5) = -4.7e-35.  Relative to the value, in u = 2^-24: the exponent -z^2/2 log2(e) takes two
    roundings and that of the constant (2.3 u, times z^2 / 2 in the exponential: 1.2 z^2 u); its exponential 2 u, the reciprocal
    2 u, the fitted factor 7 u, x 3 u, four products and the store 5 u."""
    z = -torch.linspace(0.5, 12.5, 4800, device="cuda")
    N = z.numel()
    one, zero = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(1, N, device="cuda")
    igc.linear_forward(1, N, 8, one, 8, zero, 8, Y, N, y_type=igc.IGC_F32, bias=z, act=igc.IGC_ACT_GELU, workspace=ws)
    ref = _f("gelu", z.double())[0]
    bad = ~((Y[0].double() - ref).abs() <= (20 + 1.2 * z.double() ** 2) * U * ref.abs())
    assert not bool(bad.any()), (int(bad.sum()), z[bad][:4], Y[0][bad][:4], ref[bad][:4])
