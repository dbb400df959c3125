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


@pytest.mark.parametrize("kind,x_kind", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("N", [1, 7, 41, 47, 123, 500, 511, 513, 1001, 1025, 1100, 2049, 3000, 4095, 5003, 6144, 8191, 9001, 12345, 16383, 20001, 40000,
                               70001])
def test_layer_norm_of_rows_of_one_value(torch, igc, N, kind, x_kind):  # noqa: F811
    """The value is the mean, and Y is beta: a last place of 60000 by eps^-1/2 would be more than 1."""
    values = [60000.0, -65504.0, 3.0, 0.1, 1023.5, 2.0 ** -14, 5 * 2.0 ** -24] if kind == "f16" else \
        [60000.0, 2.0 ** 65, 2.0 ** 66, -2.0 ** 100, 0.1, 1.0078125, 200.0, 3e33]
    c = torch.tensor(values, device="cuda").to(getattr(torch, {"f16": "float16", "bf16": "bfloat16"}[kind])).float()
    M = len(values)
    X = Mat(torch, M, N, x_kind, values=c[:, None].expand(M, N))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    gamma, beta = 1 + 0.3 * torch.randn(N, generator=gen, device="cuda"), torch.randn(N, generator=gen, device="cuda")
    Y = Mat(torch, M, N, kind)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    igc.layer_norm_forward(M, N, X.ptr, X.ld, Y.ptr, Y.ld, gamma=gamma, beta=beta, mean=mean, rstd=rstd,
                           type=igc.IGC_F16 if kind == "f16" else igc.IGC_BF16, x_type={"f32": igc.IGC_F32, "f16": igc.IGC_F16, "bf16": igc.IGC_BF16}[x_kind])
    assert torch.equal(mean, c), (mean - c).tolist()
    assert torch.equal(Y.t, beta.to(Y.t.dtype).expand(M, N))
    # sums of one 16-bit value (11 bits) over up to 8192 elements are exact, and the variance 0; past the registers the first
    # mean is off by up to 4 last places, and (N / 8192 + 1) 8 + 12 additions, one after the other, leave 2^-24 each of their square
    off = (4 * 2.0 ** -23 * c.double()) ** 2 * ((N // 8192 + 1) * 8 + 12) * 2.0 ** -24 if N > 16384 else 0.0 * c.double()
    ref = (off * 0 + 1e-5) ** -0.5
    assert bool(((rstd.double() / ref - 1).abs() <= 2.0 ** -22 + off / 1e-5).all()), (rstd / ref).tolist()


# Additions one after the other in a sum over a row past the registers: 512 of a thread, then fp64 sums of those, and
# 12 across the threads
DEPTH = 512 + 12


@pytest.mark.parametrize("x_kind", ["f32", "f16"])
@pytest.mark.parametrize("N", [2 ** 20 + 3, 2 ** 24 + 5])
def test_norm_of_rows_of_millions(torch, igc, ws, N, x_kind):  # noqa: F811
    """Distances far smaller than the mean, gradients of one value: what roundings of the same sign would hide."""
    U, M = 2.0 ** -24, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    noise = torch.randn(M, N, generator=gen, device="cuda")
    X = Mat(torch, M, N, x_kind, values=40.1 + (1e-3 if x_kind == "f32" else 0.1) * noise)
    del noise
    Y, mean, rstd = Mat(torch, M, N, "f16"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    kw = dict(type=igc.IGC_F16, x_type=igc.IGC_F32 if x_kind == "f32" else igc.IGC_F16)
    igc.layer_norm_forward(M, N, X.ptr, N, Y.ptr, N, mean=mean, rstd=rstd, eps=0.0, **kw)
    x = X.double()
    m = x.mean(1, keepdim=True)
    d = x - m
    var = (d * d).mean(1, keepdim=True)
    r = var ** -0.5
    first = (DEPTH + 3) * U * x.abs().mean(1, keepdim=True)                            # the first mean
    em = (DEPTH + 4) * U * (d.abs().mean(1, keepdim=True) + first) + 2 * U * m.abs()  # with that of the distances from it
    # the squares of distances from the first mean less that of its own distance, and theirs by the last mean's error
    evar = (DEPTH + 12) * U * (var + 2 * first * first) + 2 * first * em
    er = r * (0.6 * evar / var + 4 * U)
    ey = 1.1 * ((r + er) * (em + U * d.abs()) + d.abs() * er + 4 * U * d.abs() * r)
    assert float((em * r).max()) < 0.02 and float((er / r).max()) < 0.02  # (x itself is within 2e-6 of 1e-3)
    _check("mean", mean, m[:, 0], em[:, 0])
    _check("rstd", rstd, r[:, 0], er[:, 0])
    _check("Y", Y.t, d * r, ey + _store("f16", (d * r).abs() + ey))
    # the backward pass from given statistics; every g the same number, whose sums' last places round one way
    xh = x = None
    mean, rstd = m[:, 0].float(), r[:, 0].float()
    c = 1637 * 2.0 ** -14
    dY, dX = torch.full((M, N), c, dtype=torch.float16, device="cuda"), Mat(torch, M, N, x_kind)
    igc.layer_norm_backward(M, N, dY, N, X.ptr, N, mean, rstd, dX=dX.ptr, lddx=N, workspace=ws, **kw)
    xh = (X.double() - mean.double()[:, None]) * rstd.double()[:, None]
    mgx = (c * xh).mean(1, keepdim=True)
    want = rstd.double()[:, None] * (c - c - xh * mgx)
    size = (c * xh.abs()).mean(1, keepdim=True)
    ed = 1.1 * rstd.double()[:, None] * ((DEPTH + 3) * U * c + xh.abs() * (DEPTH + 6) * U * size + 6 * U * (2 * c + (xh * mgx).abs()))
    _check("dX", dX.t, want, ed + _store(x_kind, want.abs() + ed))


def test_column_sums_of_very_many_rows(torch, igc, ws):  # noqa: F811
    """2^31 rows of one gradient: 4096 additions in a thread, 2048 of workgroups' sums and a few more."""
    M, c = 2 ** 31 - 4096, 1637 * 2.0 ** -14
    dY, zeros = torch.full((M,), c, dtype=torch.float16, device="cuda"), torch.zeros(M, device="cuda")
    dgamma, dbeta = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    igc.layer_norm_backward(M, 1, dY, 1, dY, 1, zeros, zeros, dgamma=dgamma, dbeta=dbeta, type=igc.IGC_F16, workspace=ws)
    assert abs(float(dbeta) / (M * c) - 1) <= (4096 + 2048 + 80) * 2.0 ** -24 and float(dgamma) == 0.0


def test_rows_without_elements_as_torch_gives_them(torch, igc, ws):  # noqa: F811
    """Empty tensors have no address: the vectors of the rows are set all the same."""
    M = 5
    x, q = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(M, 0, dtype=torch.int8, device="cuda")
    mean, rstd, scale = (torch.full((M,), float("nan"), device="cuda") for _ in range(3))
    assert x.data_ptr() == 0
    igc.layer_norm_forward(M, 0, x, 0, x, 0, eps=0.25)
    igc.layer_norm_forward(M, 0, x, 0, x, 0, eps=0.25, mean=mean, rstd=rstd, Q=q, ldq=0, scale=scale)
    assert mean.tolist() == [0.0] * M and rstd.tolist() == [2.0] * M and scale.tolist() == [0.0] * M
    scale.fill_(float("nan"))
    igc.quantize_rows(M, 0, x, 0, q, 0, scale)
    assert scale.tolist() == [0.0] * M
    igc.layer_norm_backward(M, 0, x, 0, x, 0, mean, rstd, dX=x, lddx=0, workspace=ws)
    none = torch.empty(0, 7, dtype=torch.bfloat16, device="cuda")
    igc.layer_norm_forward(0, 7, none, 7, none, 7)
    igc.layer_norm_backward(0, 7, none, 7, none, 7, None, None, dX=none, lddx=7, workspace=ws)
    dgamma = torch.full((7,), float("nan"), device="cuda")
    igc.layer_norm_backward(0, 7, none, 7, none, 7, None, None, dX=none, lddx=7, dgamma=dgamma, workspace=ws)
    assert not bool(dgamma.any())
