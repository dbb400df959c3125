"""Few rows at an odd 2-byte offset against wide aligned weights: the rows are
copied into aligned ones first.  Against 64 bits, tolerances as in test_gpu_ffn.py."""
from __future__ import annotations

import pytest

from test_gpu_ffn import U, Mat, _check, _store, _type, igc, torch, ws  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 16, 33, 64])
def test_rows_at_odd_addresses_and_aligned_weights(torch, igc, ws, M, kind):  # noqa: F811
    N, K = 16384, 4096
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    X = Mat(torch, M, K, kind, shift=1, gen=gen)
    W, V = (Mat(torch, N, K, kind, gen=gen, std=K ** -0.5) for _ in range(2))
    Y, H = Mat(torch, M, N, kind), Mat(torch, M, N, kind)
    igc.linear_forward(M, N, K, X.ptr, K, W.ptr, K, Y.ptr, N, type=_type(igc, kind), workspace=ws)
    igc.glu_forward(M, N, K, X.ptr, K, W.ptr, K, V.ptr, K, H.ptr, N, type=_type(igc, kind), act=igc.IGC_ACT_RELU, workspace=ws)
    g, u = (X.double() @ w.double().T for w in (W, V))
    eg, eu = ((K + 2) * U * (X.double().abs() @ w.double().abs().T) for w in (W, V))
    _check("Y", Y.t, g, eg + _store(kind, g.abs() + eg))
    ref = g.clamp(min=0) * u
    e = eg * (u.abs() + eu) + g.abs() * eu + 4 * U * ref.abs()
    _check("H", H.t, ref, e + _store(kind, ref.abs() + e))
    assert Y.others_untouched() and H.others_untouched()
