"""Layer norm and rows in 8 bits on the GPU against their formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24): every sum over a row of N runs
over at most D = N / 64 + 30 additions one after the other (a thread's share,
then the threads), so it is off by D u times the sum of what it adds; other
fp32 operations by u of their result each; a store by half a step of the type.
Sums down M rows are off by at most (M + 20) u times what they add, in any
order.  Rows in 8 bits are exact.
"""
from __future__ import annotations

import pytest

from test_gpu_ffn import Mat, U, _check, _store, _type, igc, torch, ws  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-5


class Bytes:
    """rows x cols of int8 inside a value that no kernel leaves by chance everywhere."""

    def __init__(self, torch, rows, cols, ld=None, shift=0):  # noqa: F811
        self.rows, self.cols, self.ld = rows, cols, cols if ld is None else ld
        self.flat = torch.full((shift + rows * self.ld + 64,), -128, dtype=torch.int8, device="cuda")  # (-128 is no value of a row)
        self.t = self.flat[shift:shift + rows * self.ld].view(rows, self.ld)[:, :cols]
        self.ptr = self.flat.data_ptr() + shift

    def others_untouched(self):
        return int((self.flat == -128).sum()) == self.flat.numel() - self.rows * self.cols


# (M, N, extra row length, shift of the start in elements): every kernel by N, ends inside chunks, odd rows
SIZES = [(1, 1, 0, 0), (3, 5, 2, 1), (1, 8, 0, 0), (5, 64, 0, 8), (70, 65, 0, 0), (4, 511, 0, 0), (33, 512, 8, 0), (9, 513, 1, 3), (257, 1000, 0, 0),
         (6, 2048, 0, 0), (5, 2049, 0, 0), (7, 2056, 8, 8), (131, 4096, 0, 0), (3, 5001, 0, 0), (66, 8192, 0, 0), (2, 8193, 0, 2), (5, 8200, 0, 0),
         (3, 16384, 0, 0), (4, 20001, 7, 0), (2, 32768, 0, 0), (3, 32769, 0, 0), (2, 40000, 0, 0), (2, 65537, 1, 1), (1, 200000, 0, 0)]
TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")]


def _stream(torch, gen, M, N):  # noqa: F811
    """Rows of different sizes and offsets: deviations far smaller than the mean, far larger, and rows of one value."""
    x = torch.randn(M, N, generator=gen, device="cuda")
    size = torch.tensor([1.0, 0.01, 30.0, 1.0, 0.0], device="cuda").repeat(M // 5 + 1)[:M, None]
    mean = torch.tensor([0.0, 1.0, -5.0, 40.0, 3.0], device="cuda").repeat(M // 5 + 1)[:M, None]
    return x * size + mean


def _depth(n):
    return n / 64 + 30


def _norm_reference(x, gamma, beta, eps=EPS):
    """y, mean, rstd in 64 bits and how far fp32 may be off."""
    n = x.shape[1]
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    em = (_depth(n) + 3) * U * x.abs().mean(1, keepdim=True)
    evar = (_depth(n) + 8) * U * var + em * em + 2 * U * em * d.abs().mean(1, keepdim=True)
    er = rstd * (0.5 * evar / (var + eps) + 4 * U)
    g = gamma if gamma is not None else 1.0
    b = beta if beta is not None else 0.0
    y = d * rstd * g + b
    ga = abs(g)
    ey = 1.1 * (ga * (rstd + er) * (em + U * d.abs()) + d.abs() * er * ga + 4 * U * (d.abs() * rstd * ga + abs(b)))
    return y, mean[:, 0], rstd[:, 0], 1.1 * ey, 1.1 * em[:, 0], 1.1 * er[:, 0]


def _exact_rows(x):
    """Rows in 8 bits: the quotient of 16-bit values by the largest, times 127, is exact enough in 64 bits to tell every tie."""
    import torch

    top = x.abs().amax(1, keepdim=True) if x.shape[1] else x.new_zeros(x.shape[0], 1)
    q = torch.where(top > 0, (127 * x / top).round(), torch.zeros_like(x))
    return q, (top / 127).float()[:, 0]


@pytest.mark.parametrize("kind,x_kind", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_layer_norm_forward(torch, igc, size, kind, x_kind):  # noqa: F811
    M, N, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(SIZES.index(size))
    X = Mat(torch, M, N, x_kind, N + more, shift, values=_stream(torch, gen, M, N))
    for affine, outs in ((True, "ysq"), (False, "yq"), (True, "q")):
        gamma = 1 + 0.3 * torch.randn(N, generator=gen, device="cuda") if affine else None
        beta = torch.randn(N, generator=gen, device="cuda") if affine else None
        Y = Mat(torch, M, N, kind, N + more, shift)
        Q = Bytes(torch, M, N, N + more, shift)
        mean, rstd, scale = (torch.full((M + 1,), float("nan"), device="cuda") for _ in range(3))
        igc.layer_norm_forward(M, N, X.ptr, X.ld, Y.ptr if "y" in outs else None, Y.ld, gamma=gamma, beta=beta, eps=EPS,
                               mean=mean if "s" in outs else None, rstd=rstd if "s" in outs else None, Q=Q.ptr if "q" in outs else None,
                               ldq=Q.ld, scale=scale, type=_type(igc, kind), x_type=_type(igc, x_kind))
        torch.cuda.synchronize()
        y, m, r, ey, em, er = _norm_reference(X.double(), gamma.double() if affine else None, beta.double() if affine else None)
        if "y" in outs:
            _check("Y", Y.t, y, ey + _store(kind, y.abs() + ey))
            assert Y.others_untouched()
            kept = Y.t.clone()
            if "q" in outs:
                q, s = _exact_rows(Y.double())
                assert torch.equal(Q.t.double(), q) and torch.equal(scale[:M], s) and Q.others_untouched()
                assert bool(scale[M].isnan())
        if "s" in outs:
            _check("mean", mean[:M], m, em + U * m.abs())
            _check("rstd", rstd[:M], r, er)
            assert bool(mean[M].isnan()) and bool(rstd[M].isnan())
        if outs == "ysq":
            first = (kept, Q.t.clone(), scale[:M].clone(), gamma, beta)
        if outs == "q":  # alone: the rows that Y would have had
            igc.layer_norm_forward(M, N, X.ptr, X.ld, Y.ptr, Y.ld, gamma=gamma, beta=beta, eps=EPS, type=_type(igc, kind), x_type=_type(igc, x_kind))
            q, s = _exact_rows(Y.double())
            assert torch.equal(Q.t.double(), q) and torch.equal(scale[:M], s) and Q.others_untouched()
    # the same call gives the same bits
    kept, q, s, gamma, beta = first
    igc.layer_norm_forward(M, N, X.ptr, X.ld, Y.ptr, Y.ld, gamma=gamma, beta=beta, eps=EPS, Q=Q.ptr, ldq=Q.ld, scale=scale, type=_type(igc, kind),
                           x_type=_type(igc, x_kind))
    assert torch.equal(Y.t, kept) and torch.equal(Q.t, q) and torch.equal(scale[:M], s)


@pytest.mark.parametrize("kind,x_kind", TYPES, ids=str)
@pytest.mark.parametrize("N", [2049, 2500, 4096, 4100, 5001, 8192])
def test_layer_norm_forward_of_many_rows(torch, igc, N, kind, x_kind):  # noqa: F811
    """Rows enough that a workgroup takes several, with the kernels that only many rows take."""
    M = 2100
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    X = Mat(torch, M, N, x_kind, values=_stream(torch, gen, M, N))
    gamma, beta = 1 + 0.3 * torch.randn(N, generator=gen, device="cuda"), torch.randn(N, generator=gen, device="cuda")
    Y, Q, R = Mat(torch, M, N, kind), Bytes(torch, M, N), Bytes(torch, M, N)
    mean, rstd, s, t = (torch.empty(M, device="cuda") for _ in range(4))
    kw = dict(gamma=gamma, beta=beta, eps=EPS, type=_type(igc, kind), x_type=_type(igc, x_kind))
    igc.layer_norm_forward(M, N, X.ptr, N, Y.ptr, N, mean=mean, rstd=rstd, Q=Q.ptr, ldq=N, scale=s, **kw)
    y, m, r, ey, em, er = _norm_reference(X.double(), gamma.double(), beta.double())
    _check("Y", Y.t, y, ey + _store(kind, y.abs() + ey))
    _check("mean", mean, m, em + U * m.abs())
    _check("rstd", rstd, r, er)
    q, scale = _exact_rows(Y.double())
    assert torch.equal(Q.t.double(), q) and torch.equal(s, scale) and Q.others_untouched() and Y.others_untouched()
    igc.layer_norm_forward(M, N, X.ptr, N, None, N, Q=R.ptr, ldq=N, scale=t, **kw)
    assert torch.equal(R.t, Q.t) and torch.equal(s, t)
    mean.fill_(float("nan"))
    igc.layer_norm_forward(M, N, X.ptr, N, None, N, mean=mean, **kw)  # the means alone
    _check("mean", mean, m, em + U * m.abs())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_quantize_rows(torch, igc, size, kind):  # noqa: F811
    M, N, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(100 + SIZES.index(size))
    x = _stream(torch, gen, M, N)
    X = Mat(torch, M, N, kind, N + more, shift, values=x)
    Q = Bytes(torch, M, N, N + more, shift)
    scale = torch.full((M + 1,), float("nan"), device="cuda")
    igc.quantize_rows(M, N, X.ptr, X.ld, Q.ptr, Q.ld, scale, type=_type(igc, kind))
    torch.cuda.synchronize()
    q, s = _exact_rows(X.double())
    assert torch.equal(Q.t.double(), q) and torch.equal(scale[:M], s) and Q.others_untouched() and bool(scale[M].isnan())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_quantize_rows_every_quotient(torch, igc, kind):  # noqa: F811
    """Every significand by every largest significand, at distances where the quotient is 0.4 to 127: all ties among them."""
    bits = 11 if kind == "f16" else 8
    low = 2 ** (bits - 1)
    sig = torch.arange(low, 2 * low, device="cuda", dtype=torch.float32) / low  # [1, 2)
    for shift in (0, 1, 2, 3, 4, 5, 6, 7, 8):
        M = low
        x = torch.empty(M, 2 * low + 1, device="cuda")
        x[:, 0] = sig  # each row's largest, for shift 0 with smaller ones only
        x[:, 1:low + 1] = sig[None, :] * 2.0 ** -shift
        x[:, low + 1:] = -x[:, 1:low + 1]
        if shift == 0:
            x[:, 1:] = torch.where(x[:, 1:].abs() <= sig[:, None], x[:, 1:], torch.zeros_like(x[:, 1:]))
        X = x.to(torch.float16 if kind == "f16" else torch.bfloat16)
        assert torch.equal(X.float(), x)
        Q, scale = torch.empty(M, 2 * low + 1, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        igc.quantize_rows(M, 2 * low + 1, X, 2 * low + 1, Q, 2 * low + 1, scale, type=_type(igc, kind))
        q, s = _exact_rows(X.double())
        assert torch.equal(Q.double(), q) and torch.equal(scale, s)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("N", [7, 256, 3000, 40000, 70000])
def test_quantize_rows_ends_of_the_range(torch, igc, kind, N):  # noqa: F811
    """Rows of zeros, of the smallest and the largest values, with infinities and NaN."""
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    info = torch.finfo(dt)
    tiny = 2.0 ** -24 if kind == "f16" else 2.0 ** -133  # the smallest value of the type
    tops = [0.0, tiny, 3 * tiny, info.tiny, info.max, -info.max, info.max / 3, 1.0]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    X = torch.empty(len(tops) + 4, N, dtype=dt, device="cuda")
    for i, top in enumerate(tops):
        X[i] = (torch.randint(-64, 65, (N,), generator=gen, device="cuda").double() / 64 * top).to(dt)
        X[i, N // 2] = top
    X[len(tops):] = torch.randn(4, N, generator=gen, device="cuda").to(dt)
    for i, v in enumerate((float("inf"), float("-inf"), float("nan"))):
        X[len(tops) + i, N - 1 - i] = v
    X[len(tops) + 3, 0], X[len(tops) + 3, N - 1] = float("inf"), float("nan")
    M = X.shape[0]
    Q, scale = torch.full((M, N), -128, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    igc.quantize_rows(M, N, X, N, Q, N, scale, type=_type(igc, kind))
    q, s = _exact_rows(X[:len(tops)].double())
    assert torch.equal(Q[:len(tops)].double(), q) and torch.equal(scale[:len(tops)], s)
    assert bool(scale[len(tops):].isnan().all()) and not bool(Q[len(tops):].any())


def test_rows_of_no_elements(torch, igc):  # noqa: F811
    s, mean, rstd = (torch.full((4,), float("nan"), device="cuda") for _ in range(3))
    x = torch.empty(16, device="cuda")
    igc.quantize_rows(3, 0, x, 0, x, 0, s)
    assert s[:3].tolist() == [0.0] * 3 and bool(s[3].isnan())
    s.fill_(float("nan"))
    igc.layer_norm_forward(3, 0, x, 0, x, 0, mean=mean, rstd=rstd, Q=x, ldq=0, scale=s, eps=0.25)
    assert s[:3].tolist() == [0.0] * 3 and mean[:3].tolist() == [0.0] * 3 and rstd[:3].tolist() == [2.0] * 3
    assert all(bool(t[3].isnan()) for t in (s, mean, rstd))


@pytest.mark.parametrize("N", [5, 700, 5000, 33000])
def test_layer_norm_of_rows_that_are_not_finite(torch, igc, N):  # noqa: F811
    """One infinity or NaN makes its own row NaN, and no other."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    X = torch.randn(6, N, generator=gen, device="cuda").half()
    good = X.clone()
    X[1, N - 1], X[3, 0], X[4, N // 2] = float("inf"), float("nan"), float("-inf")
    Y, W = torch.empty_like(X), torch.empty_like(X)
    Q, V = (torch.full((6, N), -128, dtype=torch.int8, device="cuda") for _ in range(2))
    s, t = (torch.empty(6, device="cuda") for _ in range(2))
    igc.layer_norm_forward(6, N, X, N, Y, N, Q=Q, ldq=N, scale=s, type=igc.IGC_F16)
    igc.layer_norm_forward(6, N, good, N, W, N, Q=V, ldq=N, scale=t, type=igc.IGC_F16)
    for i in range(6):
        if i in (1, 3, 4):
            assert bool(Y[i].isnan().all()) and bool(s[i].isnan()) and not bool(Q[i].any())
        else:
            assert torch.equal(Y[i], W[i]) and torch.equal(Q[i], V[i]) and s[i] == t[i]


def _back_reference(dy, x, mean, rstd, gamma, r):
    """dx, dgamma, dbeta in 64 bits and how far fp32 may be off; mean and rstd are inputs."""
    M, n = x.shape
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma if gamma is not None else dy
    mg, mgx = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    e1 = (_depth(n) + 3) * U * g.abs().mean(1, keepdim=True)
    e2 = (_depth(n) + 6) * U * (g * xh).abs().mean(1, keepdim=True)
    dx = rstd[:, None] * (g - mg - xh * mgx)
    ed = rstd[:, None] * (e1 + xh.abs() * e2 + 6 * U * (g.abs() + mg.abs() + (xh * mgx).abs()))
    if r is not None:
        dx = dx + r
        ed = ed + 2 * U * dx.abs()
    return (dx, (dy * xh).sum(0), dy.sum(0), 1.1 * ed, 1.1 * (M + 24) * U * (dy * xh).abs().sum(0), 1.1 * (M + 20) * U * dy.abs().sum(0))


@pytest.mark.parametrize("kind,x_kind", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES + [(600, 264, 0, 0), (1500, 1001, 0, 0), (2100, 4096, 0, 0), (300, 9001, 0, 0), (1100, 16384, 0, 0)], ids=str)
def test_layer_norm_backward(torch, igc, ws, size, kind, x_kind):  # noqa: F811
    M, N, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(200 + M + N)
    x = _stream(torch, gen, M, N)
    X = Mat(torch, M, N, x_kind, N + more, shift, values=x)
    dY = Mat(torch, M, N, kind, N + more, shift, gen)
    R = Mat(torch, M, N, x_kind, N + more, shift, gen)
    xd = X.double()
    mean = xd.mean(1).float()
    rstd = (1 / (xd.var(1, unbiased=False) + EPS).sqrt()).float()
    gamma = 1 + 0.3 * torch.randn(N, generator=gen, device="cuda")
    for want, affine, residual in (("xgb", True, True), ("xgb", False, False), ("x", True, False), ("gb", True, True), ("g", False, False),
                                   ("xb", True, True)):
        dX = Mat(torch, M, N, x_kind, N + more, shift)
        dg, db = (torch.full((N + 1,), float("nan"), device="cuda") for _ in range(2))
        kw = dict(gamma=gamma if affine else None, R=R.ptr if residual else None, ldr=R.ld, dX=dX.ptr if "x" in want else None, lddx=dX.ld,
                  dgamma=dg if "g" in want else None, dbeta=db if "b" in want else None, type=_type(igc, kind), x_type=_type(igc, x_kind))
        args = (M, N, dY.ptr, dY.ld, X.ptr, X.ld, mean, rstd)
        need = igc.layer_norm_backward_workspace_size(*args, **kw)
        assert need <= ws.numel()
        ws[need:need + 256] = 255
        igc.layer_norm_backward(*args, **kw, workspace=ws)
        torch.cuda.synchronize()
        assert bool((ws[need:need + 256] == 255).all())
        dx, g, b, ex, eg, eb = _back_reference(dY.double(), xd, mean.double(), rstd.double(), gamma.double() if affine else None,
                                               R.double() if residual else None)
        if "x" in want:
            _check("dX", dX.t, dx, ex + _store(x_kind, dx.abs() + ex))
            assert dX.others_untouched()
        if "g" in want:
            _check("dgamma", dg[:N], g, eg + U * g.abs())
        if "b" in want:
            _check("dbeta", db[:N], b, eb + U * b.abs())
        assert bool(dg[N].isnan()) and bool(db[N].isnan())
        if want == "xgb" and affine:
            before = dX.t.clone(), dg.clone(), db.clone()
            igc.layer_norm_backward(*args, **kw, workspace=ws)
            assert torch.equal(before[0], dX.t) and torch.equal(before[1][:N], dg[:N]) and torch.equal(before[2][:N], db[:N])


def test_layer_norm_backward_of_no_rows(torch, igc):  # noqa: F811
    dg, db = (torch.full((300,), float("nan"), device="cuda") for _ in range(2))
    x = torch.empty(16, device="cuda")
    igc.layer_norm_backward(0, 299, x, 299, x, 299, None, None, dgamma=dg, dbeta=db)
    assert not bool(dg[:299].any()) and not bool(db[:299].any()) and bool(dg[299].isnan()) and bool(db[299].isnan())


def test_layer_norm_gradient_against_differences(torch, igc, ws):  # noqa: F811
    """dX, dgamma and dbeta against central differences of sum(dY y) in 64 bits."""
    M, N = 5, 23
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    X, dY = torch.randn(M, N, generator=gen, device="cuda") * 2 + 1, torch.randn(M, N, generator=gen, device="cuda").half()
    gamma, beta = 1 + 0.3 * torch.randn(N, generator=gen, device="cuda"), torch.randn(N, generator=gen, device="cuda")
    Y, mean, rstd = torch.empty_like(dY), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    kw = dict(type=igc.IGC_F16, x_type=igc.IGC_F32)
    igc.layer_norm_forward(M, N, X, N, Y, N, gamma=gamma, beta=beta, mean=mean, rstd=rstd, **kw)
    dX, dg, db = torch.empty_like(X), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    igc.layer_norm_backward(M, N, dY, N, X, N, mean, rstd, gamma=gamma, dX=dX, lddx=N, dgamma=dg, dbeta=db, workspace=ws, **kw)

    def loss(x, g, b):
        d = x - x.mean(1, keepdim=True)
        return (dY.double() * (d / ((d * d).mean(1, keepdim=True) + 1e-5).sqrt() * g + b)).sum()

    at = [X.double(), gamma.double(), beta.double()]
    h = 1e-5
    for which, got in ((0, dX), (1, dg), (2, db)):
        for i in range(got.numel()):
            v = []
            for sign in (1, -1):
                moved = [t.clone() for t in at]
                moved[which].view(-1)[i] += sign * h
                v.append(loss(*moved))
            diff = float(v[0] - v[1]) / (2 * h)
            # the difference: h^2 times a third derivative of at most about 100 terms, and 1e-16 of a loss of about 100 over h
            assert abs(float(got.view(-1)[i]) - diff) <= 2e-6 + 40 * U * (abs(diff) + float(dY.abs().max()) * N), (which, i)


@pytest.mark.parametrize("N", [7, 9, 60, 500, 1001, 3000, 8001, 9001, 20001])
def test_norm_of_rows_of_one_huge_value(torch, igc, ws, N):  # noqa: F811
    """Deviations of nothing, far from zero: what lies past the row in the last chunk must not come in."""
    M = 3
    X = torch.tensor([2.0 ** 100, -(2.0 ** 110), 2.0 ** 126], device="cuda")[:, None].repeat(1, N)
    X[2] = torch.where(torch.arange(N, device="cuda") % 2 == 0, X[2], -X[2])  # mean 0 or a few, deviations that overflow
    Y, mean, rstd = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    kw = dict(type=igc.IGC_BF16, x_type=igc.IGC_F32)
    igc.layer_norm_forward(M, N, X, N, Y, N, mean=mean, rstd=rstd, **kw)
    # whole powers of two: the means are off by their sums' roundings at most
    assert float((mean[:2].double() - X[:2, 0].double()).abs().max() / 2.0 ** 110) <= _depth(N) * U
    assert float(rstd[2]) == 0.0 and not bool(Y[2].any())  # (the variance is past fp32: as the formula has it there)
    mean[:2] = X[:2, 0]
    rstd[:2] = 316.0
    dY = torch.randn(M, N, device="cuda").bfloat16()
    dX, dg, db = torch.empty_like(X), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    igc.layer_norm_backward(2, N, dY, N, X, N, mean, rstd, dX=dX, lddx=N, dgamma=dg, dbeta=db, workspace=ws, **kw)
    d = dY[:2].double()
    want = 316.0 * (d - d.mean(1, keepdim=True))
    assert float((dX[:2].double() - want).abs().max()) <= 316.0 * (_depth(N) + 4) * U * float(d.abs().max()) * 2
    assert not bool(dg.any())


def test_rows_past_32_bit_offsets(torch, igc, ws):  # noqa: F811
    """Rows that begin more than 2^32 bytes, and 2^31 elements, into their matrices."""
    M, N, ld = 3, 520, 2 ** 30 + 64
    flat = torch.empty(2 * ld + N, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2 * ld + N, dtype=torch.bfloat16, device="cuda")
    q = torch.full((2 * ld + N,), -128, dtype=torch.int8, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    rows, outs = torch.as_strided(flat, (M, N), (ld, 1)), torch.as_strided(out, (M, N), (ld, 1))
    qs = torch.as_strided(q, (M, N), (ld, 1))
    rows.copy_(x)
    want, s, t = torch.empty_like(x), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    q1 = torch.empty(M, N, dtype=torch.int8, device="cuda")
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    igc.layer_norm_forward(M, N, flat, ld, out, ld, Q=q, ldq=ld, scale=s, mean=mean, rstd=rstd)
    igc.layer_norm_forward(M, N, x, N, want, N, Q=q1, ldq=N, scale=t)
    assert torch.equal(outs, want) and torch.equal(qs, q1) and torch.equal(s, t)
    igc.quantize_rows(M, N, flat, ld, q, ld, s)
    igc.quantize_rows(M, N, x, N, q1, N, t)
    assert torch.equal(qs, q1) and torch.equal(s, t)
    dy = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    dx, dg, dg1 = torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    igc.layer_norm_backward(M, N, dy, N, flat, ld, mean, rstd, R=flat, ldr=ld, dX=out, lddx=ld, dgamma=dg, workspace=ws)
    igc.layer_norm_backward(M, N, dy, N, x, N, mean, rstd, R=x, ldr=N, dX=dx, lddx=N, dgamma=dg1, workspace=ws)
    assert torch.equal(outs, dx) and torch.equal(dg, dg1)
    igc.dropout(M, N, flat, ld, out, ld, 0.3, 5, R=flat, ldr=ld)
    igc.dropout(M, N, x, N, dx, N, 0.3, 5, R=x, ldr=N)
    assert torch.equal(outs, dx)


@pytest.mark.parametrize("kind,x_kind", TYPES, ids=str)
@pytest.mark.parametrize("N", [20001, 33001])
def test_layer_norm_forward_of_many_long_rows(torch, igc, N, kind, x_kind):  # noqa: F811
    """Rows that are read again, several to a workgroup, one and two workgroups to a compute unit."""
    test_layer_norm_forward_of_many_rows(torch, igc, N, kind, x_kind)


@pytest.mark.parametrize("kind,x_kind", TYPES, ids=str)
@pytest.mark.parametrize("size", [(900, 8193, 1, 1), (1700, 8207, 0, 0), (800, 12290, 3, 1)], ids=str)
def test_layer_norm_backward_of_many_long_rows(torch, igc, ws, size, kind, x_kind):  # noqa: F811
    """Rows by columns, the next row and the next chunk on their way, with a last chunk of 1 to 7 elements."""
    test_layer_norm_backward(torch, igc, ws, size, kind, x_kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("N", [2049, 2500, 4095, 4096])
def test_layer_norm_forward_of_thousands_of_rows(torch, igc, N, kind):  # noqa: F811
    """fp32 rows enough for two chunks a thread, with statistics, in 8 bits, and the same rows a few at a time."""
    M, few = 4200, 300
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    X = Mat(torch, M, N, "f32", N + 1, values=_stream(torch, gen, M, N))
    gamma, beta = 1 + 0.3 * torch.randn(N, generator=gen, device="cuda"), torch.randn(N, generator=gen, device="cuda")
    Y, Q = Mat(torch, M, N, kind, N + 3), Bytes(torch, M, N)
    mean, rstd, s = (torch.empty(M, device="cuda") for _ in range(3))
    kw = dict(gamma=gamma, beta=beta, eps=EPS, type=_type(igc, kind), x_type=igc.IGC_F32)
    igc.layer_norm_forward(M, N, X.ptr, X.ld, Y.ptr, Y.ld, mean=mean, rstd=rstd, Q=Q.ptr, ldq=N, scale=s, **kw)
    y, m, r, ey, em, er = _norm_reference(X.double(), gamma.double(), beta.double())
    _check("Y", Y.t, y, ey + _store(kind, y.abs() + ey))
    _check("mean", mean, m, em + U * m.abs())
    _check("rstd", rstd, r, er)
    q, scale = _exact_rows(Y.double())
    assert torch.equal(Q.t.double(), q) and torch.equal(s, scale) and Q.others_untouched() and Y.others_untouched()
    V = Mat(torch, few, N, kind)
    igc.layer_norm_forward(few, N, X.ptr, X.ld, V.ptr, V.ld, **kw)
    _check("Y of few", V.t, y[:few], (ey + _store(kind, y.abs() + ey))[:few])
