"""The row operators at the ends of their numbers' ranges: rows whose squares pass
fp32 where their distances do not.  Tolerances as in test_gpu_rows.py."""
from __future__ import annotations

import pytest

from test_gpu_ffn import Mat, _check, _store, igc, torch, ws  # noqa: F401
from test_gpu_rows import Bytes, _exact_rows, _norm_reference

pytestmark = pytest.mark.gpu

# rows by 2, 4, 8 and 16 waves, the last ones of them past the row (or not: 1024, 2048, 4096, 8192); two chunks a thread; read again
LENGTHS = [1000, 1024, 1025, 1100, 1200, 1536, 2048, 2049, 2500, 3000, 3584, 4096, 4097, 5001, 5120, 6144, 7680, 8192, 9001, 20001]


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("N", LENGTHS)
def test_layer_norm_forward_far_from_zero(torch, igc, N, x_kind):  # noqa: F811
    """Means whose squares pass fp32, distances from them whose squares do not: by the formula, whatever the length."""
    M = 5
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    # |mean| > 2^64; squares of distances of up to 2e34 (bf16, whose steps are 1.4e17 there) by N <= 8192 elements, or of
    # 1e32 by more, stay below 3.4e38 in their sums
    size = 7.5e15 if x_kind == "f32" else 1.2e17 if N <= 8192 else 7e16
    mean = torch.tensor([2.0e19, -2.0e19, 2.5e19, -3.0e19, 2.0e19], device="cuda")[:, None]
    X = Mat(torch, M, N, x_kind, values=mean + size * torch.randn(M, N, generator=gen, device="cuda"))
    gamma, beta = 1 + 0.3 * torch.randn(N, generator=gen, device="cuda"), torch.randn(N, generator=gen, device="cuda")
    Y, Q = Mat(torch, M, N, "bf16"), Bytes(torch, M, N)
    m, r, s = (torch.empty(M, device="cuda") for _ in range(3))
    igc.layer_norm_forward(M, N, X.ptr, X.ld, Y.ptr, Y.ld, gamma=gamma, beta=beta, mean=m, rstd=r, Q=Q.ptr, ldq=N, scale=s, type=igc.IGC_BF16,
                           x_type=igc.IGC_F32 if x_kind == "f32" else igc.IGC_BF16)
    y, mean, rstd, ey, em, er = _norm_reference(X.double(), gamma.double(), beta.double())
    assert float((er / rstd).max()) < 0.2 and float(ey.max()) < 2.0  # (the tolerance tells a norm from none)
    _check("mean", m, mean, em + 2.0 ** -24 * mean.abs())
    _check("rstd", r, rstd, er)
    _check("Y", Y.t, y, ey + _store("bf16", y.abs() + ey))
    q, scale = _exact_rows(Y.double())
    assert torch.equal(Q.t.double(), q) and torch.equal(s, scale) and Y.others_untouched() and Q.others_untouched()
