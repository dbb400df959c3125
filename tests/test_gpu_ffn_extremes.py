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
