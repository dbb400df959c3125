"""The feed-forward operators' backward passes over the whole range of fp16, on
the GPU against their formulas in 64 bits.

D = dY act'(Z) (dG and dU of the gated block) leaves the range of fp16 where
every input and every gradient is inside it: dY is small and the sums over many
rows are not, or dH U is large and the weights are not.

Tolerances (u = 2^-24, e = half a step of fp16 relative to the value, 2^-11):
 - D in fp32: 8 u |dY| (1 + |Z|) (times 1 + |U| for dG), as in test_gpu_ffn.py;
 - D scaled by a power of two and rounded to fp16: e |D|, and for elements so
   small that they become subnormal half of fp16's smallest step 2^-24 at that
   scale: 2^-25 / 2^10 where the largest |D| is in [2^-18, 2^5); elsewhere the
   scale takes the largest |D| to [2^14, 2^15): 2^-25 / 2^14 of it;
 - the sums over r terms in fp32: (r + 2) u sum |a b|;
 - the store: e |value| and half of fp16's smallest step.
"""
from __future__ import annotations

import pytest

from test_gpu_ffn import U, Mat, _act_id, _check, _f, _store, igc, torch, ws  # noqa: F401

pytestmark = pytest.mark.gpu

HALF16 = 2.0 ** -11


def _rounded(d, ed, most):
    """How far D may be off after its rounding."""
    most = float(most)
    step = 2.0 ** -35 if 2.0 ** -18 <= most < 2.0 ** 5 else 2.0 ** -39 * most
    return ed + HALF16 * 1.001 * (d.abs() + ed) + 1.001 * step


def _product(name, got, a, ea, b, way):
    """got = a b (way "x") or a^T b (way "w"), the elements of a off by ea."""
    if way == "w":
        a, ea = a.T, ea.T
    r = a.shape[1]
    ref, s = a @ b, a.abs() @ b.abs()
    e = ea @ b.abs() + (r + 2) * U * s
    _check(name, got, ref, e + _store("f16", ref.abs() + e))
    return ref


def _linear(torch, igc, ws, size, act, std, want="xwb", wstd=None):  # noqa: F811
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6000 + M)
    mat = lambda r, c, s: Mat(torch, r, c, "f16", c + more, shift, gen, s)  # noqa: E731
    dY, Z, X, W = mat(M, N, std), mat(M, N, 1.5), mat(M, K, 1.0), mat(N, K, K ** -0.5 if wstd is None else wstd)
    dX, dW = Mat(torch, M, K, "f16", K + more, shift), Mat(torch, N, K, "f16", K + more, shift)
    db = torch.empty(N, device="cuda")
    kw = dict(Z=Z.ptr if act != "none" else None, ldz=Z.ld, X=X.ptr, ldx=X.ld, W=W.ptr, ldw=W.ld, dX=dX.ptr if "x" in want else None,
              lddx=dX.ld, dW=dW.ptr if "w" in want else None, lddw=dW.ld, dbias=db if "b" in want else None, type=igc.IGC_F16,
              act=_act_id(igc, act))
    assert igc.linear_backward_workspace_size(M, N, K, dY.ptr, dY.ld, **kw) <= ws.numel()
    igc.linear_backward(M, N, K, dY.ptr, dY.ld, **kw, workspace=ws)
    torch.cuda.synchronize()
    d = dY.double() * _f(act, Z.double())[1]
    ed = 8 * U * dY.double().abs() * (1 + Z.double().abs())
    er = ed if act == "none" else _rounded(d, ed, d.abs().max())
    if "x" in want:
        _product("dX", dX.t, d, er, W.double(), "x")
        assert dX.others_untouched()
    if "w" in want:
        ref = _product("dW", dW.t, d, er, X.double(), "w")
        assert float(ref.abs().max()) > 2.0 ** -20 and dW.others_untouched()  # (there is something to see)
    if "b" in want:
        _check("db", db, d.sum(0), ed.sum(0) + (M + 2) * U * d.abs().sum(0) + 2.0 ** -150)


# whole tiles; odd rows, which are padded; rows too short to pad, by the register-staged kernel; few rows; one row
SIZES = [(2048, 264, 328, 0, 0), (2051, 257, 321, 1, 1), (4100, 72, 5, 0, 0), (40, 520, 264, 8, 0), (1, 64, 64, 0, 0)]


@pytest.mark.parametrize("std", [3e-7, 1e-6, 1e-5, 1e-2, 3000.0])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_gradients_of_any_size(torch, igc, ws, size, std):  # noqa: F811
    # large dY: weights that keep dX and dW = D^T X inside fp16 (X of 1, up to
    # 4100 rows: |dW| up to about 5 * 3000 * sqrt(4100) leaves it, so dX alone)
    want = "xwb" if std < 1 else "xb"
    if size[0] == 1 or size[2] == 5:
        want = want.replace("w", "") if size[0] == 1 else want
    _linear(torch, igc, ws, size, "silu", std, want, 2.0 ** -6 if std > 1 else None)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "sigmoid"])
def test_small_linear_gradients_of_every_activation(torch, igc, ws, act):  # noqa: F811
    _linear(torch, igc, ws, (2048, 200, 136, 0, 0), act, 1e-6)
    _linear(torch, igc, ws, (2048, 201, 137, 0, 0), act, 1e-6)


def _glu(torch, igc, ws, size, act, hstd, ustd, wstd, xstd=1.0, want="xgubc", shift=0):  # noqa: F811
    M, N, K = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7000 + M)
    mat = lambda r, c, s: Mat(torch, r, c, "f16", c, shift, gen, s)  # noqa: E731
    dH, G, Uo, X, Wg, Wu = mat(M, N, hstd), mat(M, N, 1.0), mat(M, N, ustd), mat(M, K, xstd), mat(N, K, wstd), mat(N, K, wstd)
    dX, dWg, dWu = (Mat(torch, r, K, "f16", K, shift) for r in (M, N, N))
    dbg, dbu = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    on = lambda c, v: v if c in want else None  # noqa: E731
    args = (M, N, K, dH.ptr, N, G.ptr, N, Uo.ptr, N)
    kw = dict(X=X.ptr, ldx=K, Wg=Wg.ptr, ldwg=K, Wu=Wu.ptr, ldwu=K, dX=on("x", dX.ptr), lddx=K, dWg=on("g", dWg.ptr), lddwg=K,
              dWu=on("u", dWu.ptr), lddwu=K, dbias_g=on("b", dbg), dbias_u=on("c", dbu), type=igc.IGC_F16, act=_act_id(igc, act))
    assert igc.glu_backward_workspace_size(*args, **kw) <= ws.numel()
    igc.glu_backward(*args, **kw, workspace=ws)
    torch.cuda.synchronize()
    f, slope = _f(act, G.double())
    dh, u = dH.double(), Uo.double()
    du, dg = dh * f, dh * u * slope
    eu = 8 * U * dh.abs() * (1 + G.double().abs())
    eg = eu * (1 + u.abs())
    most = max(float(dg.abs().max()), float(du.abs().max()))
    ru, rg = _rounded(du, eu, most), _rounded(dg, eg, most)
    if "x" in want:
        a, ea = torch.cat([dg, du], 1), torch.cat([rg, ru], 1) + 130 * U * torch.cat([dg, du], 1).abs()
        _product("dX", dX.t, a, ea, torch.cat([Wg.double(), Wu.double()], 0), "x")
    for c, out, d, r in (("g", dWg, dg, rg), ("u", dWu, du, ru)):
        if c in want:
            _product("dW" + c, out.t, d, r, X.double(), "w")
    for c, out, d, e in (("b", dbg, dg, eg), ("c", dbu, du, eu)):
        if c in want:
            _check("db" + c, out, d.sum(0), e.sum(0) + (M + 2) * U * d.abs().sum(0) + 2.0 ** -150)


@pytest.mark.parametrize("want", ["xgubc", "x", "gb"])
@pytest.mark.parametrize("size,shift", [((300, 200, 136), 0), ((300, 201, 137), 1), ((24, 7, 5), 0)], ids=str)
def test_gated_gradients_past_the_largest_fp16(torch, igc, ws, size, shift, want):  # noqa: F811
    # dG = dH U act'(G) of about 600 * 200 = 1.2e5, past 65504; weights and
    # inputs of 2^-13 keep dX and both dW inside
    _glu(torch, igc, ws, size, "silu", 600.0, 200.0, 2.0 ** -13, 2.0 ** -13, want, shift)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("size,shift", [((4096, 200, 136), 0), ((4097, 201, 137), 1)], ids=str)
def test_gated_gradients_under_the_smallest_fp16(torch, igc, ws, size, shift, act):  # noqa: F811
    # dG of about 2e-4 * 1e-4 = 2e-8, under half of fp16's smallest step; dU of 2e-4
    _glu(torch, igc, ws, size, act, 2e-4, 1e-4, size[2] ** -0.5, 1.0, "xgubc", shift)


def test_gradients_of_the_wide_layer(torch, igc, ws):  # noqa: F811
    """More blocks of D than workgroups that make it anew at another scale."""
    M, N, K = 16, 530000, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    dY = (torch.randn(M, N, generator=gen, device="cuda") * 1e-6).half()
    Z = torch.ones(M, N, dtype=torch.float16, device="cuda")
    dY[11, 529999] = 64.0  # the largest, past 2^5, in the last block
    X = torch.ones(M, K, dtype=torch.float16, device="cuda")
    dW = torch.empty(N, K, dtype=torch.float16, device="cuda")
    kw = dict(Z=Z, ldz=N, X=X, ldx=K, dW=dW, lddw=K, type=igc.IGC_F16, act=igc.IGC_ACT_RELU)
    big = torch.empty(igc.linear_backward_workspace_size(M, N, K, dY, N, **kw), dtype=torch.uint8, device="cuda")
    igc.linear_backward(M, N, K, dY, N, **kw, workspace=big)
    d = dY.double()
    _product("dW", dW, d, _rounded(d, 0 * d, d.abs().max()), X.double(), "w")


def test_gradients_that_are_not_finite_stay_where_they_are(torch, igc, ws):  # noqa: F811
    """Infinities and NaN in one row reach that row of dX and every element of dW, and leave the other rows of dX as exact as before."""
    M, N, K = 72, 64, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    Z = torch.randn(M, N, generator=gen, device="cuda").half()
    W = (torch.randn(N, K, generator=gen, device="cuda") * K ** -0.5).half()
    for bad in (float("inf"), float("nan")):
        dY = (torch.randn(M, N, generator=gen, device="cuda") * 1e-5).half()
        dY[5, 7] = bad
        dX = torch.empty(M, K, dtype=torch.float16, device="cuda")
        igc.linear_backward(M, N, K, dY, N, Z=Z, ldz=N, W=W, ldw=K, dX=dX, lddx=K, type=igc.IGC_F16, act=igc.IGC_ACT_SIGMOID, workspace=ws)
        rows = [i for i in range(M) if i != 5]
        assert not bool(torch.isfinite(dX[5]).any())
        d = dY[rows].double() * _f("sigmoid", Z[rows].double())[1]
        ed = 8 * U * dY[rows].double().abs() * (1 + Z[rows].double().abs())
        _product("dX", dX[rows], d, _rounded(d, ed, d.abs().max()), W.double(), "x")


def test_gradients_of_zero(torch, igc, ws):  # noqa: F811
    M, N, K = 64, 64, 64
    zero, one = (torch.full((64, 64), v, dtype=torch.float16, device="cuda") for v in (0.0, 1.0))
    dX, dW = torch.full_like(one, float("nan")), torch.full_like(one, float("nan"))
    igc.linear_backward(M, N, K, zero, N, Z=one, ldz=N, X=one, ldx=K, W=one, ldw=K, dX=dX, lddx=K, dW=dW, lddw=K, type=igc.IGC_F16,
                        act=igc.IGC_ACT_GELU, workspace=ws)
    assert int(dX.count_nonzero()) == 0 and int(dW.count_nonzero()) == 0


def test_replays_with_gradients_of_changing_size(torch, igc):  # noqa: F811
    """A captured backward pass finds D's scale anew on every replay."""
    M, N, K = 200, 333, 264
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)
    new = lambda r, c: torch.empty(r, c, dtype=torch.float16, device="cuda")  # noqa: E731
    unit, Z, G = (torch.randn(M, N, generator=gen, device="cuda") for _ in range(3))
    Z, G, dY = Z.half(), G.half(), new(M, N)
    X, W, V = ((torch.randn(r, K, generator=gen, device="cuda") * 2.0 ** -6).half() for r in (M, N, N))
    dX, dW, hX, hW, hV = new(M, K), new(N, K), new(M, K), new(N, K), new(N, K)
    space = torch.full((32 << 20,), 255, dtype=torch.uint8, device="cuda")

    def step():
        igc.linear_backward(M, N, K, dY, N, Z=Z, ldz=N, X=X, ldx=K, W=W, ldw=K, dX=dX, lddx=K, dW=dW, lddw=K, type=igc.IGC_F16,
                            act=igc.IGC_ACT_GELU, workspace=space)
        igc.glu_backward(M, N, K, dY, N, G, N, Z, N, X=X, ldx=K, Wg=W, ldwg=K, Wu=V, ldwu=K, dX=hX, lddx=K, dWg=hW, lddwg=K, dWu=hV,
                         lddwu=K, type=igc.IGC_F16, workspace=space)

    outs = [dX, dW, hX, hW, hV]
    dY.copy_(unit)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for std in (1.0, 2000.0, 1e-7, 1.0, 1e-2, 2000.0):
        dY.copy_(unit * std)
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        for g, t in zip(got, outs):
            assert bool(torch.isfinite(t).all()) and torch.equal(g, t), std
