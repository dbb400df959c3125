"""The feed-forward operators on the GPU against their formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, e = half a step of a type relative
to the value):
 - a product over r terms in fp32: r u sum |a b|; the activations, their
   slopes and the two or three fp32 operations after them: 8 u of what they
   are applied to, through a slope of at most 1.13 (forward) or of a second
   derivative of at most 0.8 (backward);
 - a store: e |value|, and half of the type's smallest step;
 - the backward products take D rounded to the operands' type: e sum |d w|.
Every input lies in rows of a longer buffer filled with NaN, and every output
in one whose other elements must stay as they were.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")


@pytest.fixture(scope="module")
def torch():
    import torch

    assert torch.cuda.is_available()
    return torch


@pytest.fixture(scope="module")
def igc(torch):
    import implicit_gemm_convolution_amd as m

    assert m.device_check() == m.IGC_OK, m.last_error()
    return m


@pytest.fixture(scope="module")
def ws(torch):
    """One workspace that every call of this file shares; NaN to begin with."""
    return torch.full((256 << 20,), 255, dtype=torch.uint8, device="cuda")


def _dt(torch, kind):
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[kind]


def _type(igc, kind):
    return {"f16": igc.IGC_F16, "bf16": igc.IGC_BF16, "f32": igc.IGC_F32}[kind]


def _act_id(igc, act):
    return getattr(igc, "IGC_ACT_" + act.upper())


class Mat:
    """rows x cols inside NaN, `shift` elements off the allocation's start."""

    def __init__(self, torch, rows, cols, kind, ld=None, shift=0, gen=None, std=1.0, values=None):
        self.ld = cols if ld is None else ld
        self.rows, self.cols = rows, cols
        self.flat = torch.full((shift + rows * self.ld + 64,), float("nan"), dtype=_dt(torch, kind), device="cuda")
        self.t = self.flat[shift:shift + rows * self.ld].view(rows, self.ld)[:, :cols] if rows and self.ld else self.flat[shift:shift]
        self.ptr = self.flat.data_ptr() + shift * self.flat.element_size()
        if rows and cols:
            if values is not None:
                self.t.copy_(values)
            elif gen is not None:
                self.t.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * std)

    def double(self):
        return self.t.double() if self.rows and self.cols else self.t.new_zeros(self.rows, self.cols).double()

    def others_untouched(self):
        """Every element outside the matrix is still NaN, and none inside is."""
        n = int(self.flat.isnan().sum())
        return n == self.flat.numel() - self.rows * self.cols


def _f(act, z):
    """The activation and its derivative."""
    import torch

    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        c = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return (z * s, s * (1 + z * (1 - s))) if act == "silu" else (s, s * (1 - s))


def _check(name, got, ref, tol):
    import torch

    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (name, int(bad.sum()), bad.numel(), float((err / tol)[bad].max()), torch.nonzero(bad)[:4].tolist())


def _store(kind, value):
    return HALF[kind] * value.abs() * 1.001 + TINY[kind]


# (M, N, K, extra row length, shift of the start in elements)
SIZES = [
    (1, 1, 1, 0, 0), (1, 16, 8, 0, 0), (3, 5, 7, 2, 1), (1, 300, 520, 0, 0), (2, 1001, 333, 0, 1), (5, 64, 0, 3, 0), (70, 64, 0, 8, 0),
    (16, 96, 2048, 0, 0), (17, 33, 65, 0, 0), (24, 520, 1000, 8, 8), (33, 130, 264, 0, 0), (63, 200, 72, 8, 0), (64, 64, 64, 0, 0),
    (65, 257, 129, 1, 3), (128, 256, 512, 0, 0), (131, 1000, 520, 0, 0), (200, 264, 328, 8, 16), (256, 512, 256, 0, 0), (300, 777, 1001, 0, 0),
    (513, 640, 192, 0, 0),
]
LARGE = [(2100, 2056, 264, 0, 0), (1025, 4104, 200, 8, 0), (4100, 1030, 136, 0, 2), (3400, 4104, 136, 0, 0), (3400, 136, 4104, 8, 8),
         (136, 3400, 4104, 0, 0), (520, 4104, 4096, 0, 0)]


def _linear_forward(torch, igc, ws, size, kind, act, bias, residual, save, y, seed=0, use_ws=True, stream=None):
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000 + seed)
    X = Mat(torch, M, K, kind, K + more, shift, gen)
    W = Mat(torch, N, K, kind, K + more, shift, gen, max(K, 1) ** -0.5)
    b = torch.randn(N, generator=gen, device="cuda") if bias else None
    R = Mat(torch, M, N, y, N + more, shift, gen) if residual else None
    Y = Mat(torch, M, N, y, N + more, shift)
    Z = Mat(torch, M, N, kind, N + more, shift) if save else None
    more_args = dict(type=_type(igc, kind), act=_act_id(igc, act), y_type=_type(igc, y), bias=b, R=R and R.ptr, ldr=N + more,
                     Z=Z and Z.ptr, ldz=N + more)
    args = (M, N, K, X.ptr, X.ld, W.ptr, W.ld, Y.ptr, Y.ld)
    need = igc.linear_forward_workspace_size(*args, **more_args)
    assert need <= ws.numel()
    igc.linear_forward(*args, **more_args, workspace=ws if use_ws else None, stream=stream)
    torch.cuda.synchronize()
    z = X.double() @ W.double().T
    s = X.double().abs() @ W.double().abs().T
    if bias:
        z, s = z + b.double(), s + b.double().abs()
    ez = (K + 2) * U * s
    f = _f(act, z)[0]
    ref = f + R.double() if residual else f
    ey = 1.13 * ez + 8 * U * (z.abs() + f.abs() + ref.abs() + 1)
    _check("Y", Y.t, ref, ey + _store(y, ref.abs() + ey))
    assert Y.others_untouched()
    if save:
        _check("Z", Z.t, z, ez + _store(kind, z.abs() + ez))
        assert Z.others_untouched()
    return Y.t.clone()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_forward(torch, igc, ws, size, kind):
    i = SIZES.index(size)
    for j in range(3):
        n = i + 7 * j
        _linear_forward(torch, igc, ws, size, kind, ACTS[n % 6], n % 2 == 0, n % 3 == 1, n % 4 != 1,
                        "f32" if n % 5 == 2 else kind, seed=n, use_ws=j != 2)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", LARGE, ids=str)
def test_linear_forward_large(torch, igc, ws, size, kind):
    _linear_forward(torch, igc, ws, size, kind, "gelu", True, True, True, "f32" if kind == "f16" else kind)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_linear_forward_activations(torch, igc, ws, act, y):
    _linear_forward(torch, igc, ws, (40, 72, 64, 0, 0), "bf16", act, True, y == "f32", True, y)


def _linear_backward(torch, igc, ws, size, kind, act, want, seed=0):
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2000 + seed)
    dY = Mat(torch, M, N, kind, N + more, shift, gen)
    Z = Mat(torch, M, N, kind, N + more, shift, gen, 1.5)
    X = Mat(torch, M, K, kind, K + more, shift, gen)
    W = Mat(torch, N, K, kind, K + more, shift, gen, max(K, 1) ** -0.5)
    dX, dW = Mat(torch, M, K, kind, K + more, shift), Mat(torch, N, K, kind, K + more, shift)
    db = torch.full((N + 1,), float("nan"), device="cuda")
    kw = dict(Z=Z.ptr if act != "none" else None, ldz=Z.ld, X=X.ptr, ldx=X.ld, W=W.ptr, ldw=W.ld,
              dX=dX.ptr if "x" in want else None, lddx=dX.ld, dW=dW.ptr if "w" in want else None, lddw=dW.ld,
              dbias=db if "b" in want else None, type=_type(igc, kind), act=_act_id(igc, act))
    args = (M, N, K, dY.ptr, dY.ld)
    need = igc.linear_backward_workspace_size(*args, **kw)
    assert need <= ws.numel()
    igc.linear_backward(*args, **kw, workspace=ws)
    torch.cuda.synchronize()
    d = dY.double() * _f(act, Z.double())[1]
    ed = 8 * U * dY.double().abs() * (1 + Z.double().abs())
    # what rounding D to the operands' type adds
    er = ed if act == "none" else ed + _store(kind, d.abs() + ed)
    if "x" in want:
        ref, s = d @ W.double(), d.abs() @ W.double().abs()
        e = er @ W.double().abs() + (N + 2) * U * s
        _check("dX", dX.t, ref, e + _store(kind, ref.abs() + e))
    if "w" in want:
        ref, s = d.T @ X.double(), d.abs().T @ X.double().abs()
        e = er.T @ X.double().abs() + (M + 2) * U * s
        _check("dW", dW.t, ref, e + _store(kind, ref.abs() + e))
    if "b" in want:
        _check("db", db[:N], d.sum(0), ed.sum(0) + (M + 2) * U * d.abs().sum(0) + TINY["f32"])
        assert bool(db[N].isnan())
    for m, w in ((dX, "x"), (dW, "w")):
        assert m.others_untouched() if w in want else bool(m.flat.isnan().all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES + LARGE, ids=str)
def test_linear_backward(torch, igc, ws, size, kind):
    i = (SIZES + LARGE).index(size)
    for j, want in enumerate(("xwb", "xw", "b", "x", "wb")):
        if j > 1 and size in LARGE:
            break
        _linear_backward(torch, igc, ws, size, kind, ACTS[(i + j) % 6], want, seed=i)


def _glu(torch, igc, ws, size, kind, act, bias, save, seed=0):
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3000 + seed)
    X = Mat(torch, M, K, kind, K + more, shift, gen)
    Wg = Mat(torch, N, K, kind, K + more, shift, gen, max(K, 1) ** -0.5)
    Wu = Mat(torch, N, K, kind, K + 2 * more, shift, gen, max(K, 1) ** -0.5)
    bg, bu = (torch.randn(N, generator=gen, device="cuda") if bias else None for _ in range(2))
    H = Mat(torch, M, N, kind, N + more, shift)
    G, Uo = (Mat(torch, M, N, kind, N + more, shift) if save else None for _ in range(2))
    kw = dict(bias_g=bg, bias_u=bu, G=G and G.ptr, ldg=N + more, U=Uo and Uo.ptr, ldu=N + more, type=_type(igc, kind),
              act=_act_id(igc, act))
    args = (M, N, K, X.ptr, X.ld, Wg.ptr, Wg.ld, Wu.ptr, Wu.ld, H.ptr, H.ld)
    assert igc.glu_forward_workspace_size(*args, **kw) <= ws.numel()
    igc.glu_forward(*args, **kw, workspace=ws)
    torch.cuda.synchronize()
    x, xa = X.double(), X.double().abs()
    g, u = x @ Wg.double().T, x @ Wu.double().T
    eg, eu = (K + 2) * U * (xa @ Wg.double().abs().T), (K + 2) * U * (xa @ Wu.double().abs().T)
    if bias:
        g, u = g + bg.double(), u + bu.double()
        eg, eu = eg + 2 * U * bg.double().abs(), eu + 2 * U * bu.double().abs()
    f = _f(act, g)[0]
    ref = f * u
    ef = 1.13 * eg + 8 * U * (g.abs() + f.abs() + 1)
    e = ef * (u.abs() + eu) + f.abs() * eu + 4 * U * ref.abs()
    _check("H", H.t, ref, e + _store(kind, ref.abs() + e))
    assert H.others_untouched()
    if save:
        _check("G", G.t, g, eg + _store(kind, g.abs() + eg))
        _check("U", Uo.t, u, eu + _store(kind, u.abs() + eu))
        assert G.others_untouched() and Uo.others_untouched()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES + LARGE, ids=str)
def test_glu_forward(torch, igc, ws, size, kind):
    i = (SIZES + LARGE).index(size)
    for j in range(2):
        _glu(torch, igc, ws, size, kind, ACTS[(i + 2 * j) % 6], (i + j) % 2 == 0, (i + j) % 3 != 0, seed=i)


def _glu_backward(torch, igc, ws, size, kind, act, want, seed=0):
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4000 + seed)
    dH, G, Uo = (Mat(torch, M, N, kind, N + more, shift, gen) for _ in range(3))
    X = Mat(torch, M, K, kind, K + more, shift, gen)
    Wg, Wu = (Mat(torch, N, K, kind, K + more, shift, gen, max(K, 1) ** -0.5) for _ in range(2))
    dX, dWg, dWu = Mat(torch, M, K, kind, K + more, shift), Mat(torch, N, K, kind, K + more, shift), Mat(torch, N, K, kind, K + more, shift)
    dbg, dbu = (torch.full((N + 1,), float("nan"), device="cuda") for _ in range(2))
    on = lambda c, v: v if c in want else None  # noqa: E731
    kw = dict(X=X.ptr, ldx=X.ld, Wg=Wg.ptr, ldwg=Wg.ld, Wu=Wu.ptr, ldwu=Wu.ld, dX=on("x", dX.ptr), lddx=dX.ld,
              dWg=on("g", dWg.ptr), lddwg=dWg.ld, dWu=on("u", dWu.ptr), lddwu=dWu.ld, dbias_g=on("b", dbg), dbias_u=on("c", dbu),
              type=_type(igc, kind), act=_act_id(igc, act))
    args = (M, N, K, dH.ptr, dH.ld, G.ptr, G.ld, Uo.ptr, Uo.ld)
    assert igc.glu_backward_workspace_size(*args, **kw) <= ws.numel()
    igc.glu_backward(*args, **kw, workspace=ws)
    torch.cuda.synchronize()
    f, slope = _f(act, G.double())
    dh = dH.double()
    du, dg = dh * f, dh * Uo.double() * slope
    base = 8 * U * dh.abs() * (1 + G.double().abs())
    eu, eg = base, base * (1 + Uo.double().abs())
    ru, rg = eu + _store(kind, du.abs() + eu), eg + _store(kind, dg.abs() + eg)
    if "x" in want:
        ref = dg @ Wg.double() + du @ Wu.double()
        e = (rg + (2 * N + 130) * U * dg.abs()) @ Wg.double().abs() + (ru + (2 * N + 130) * U * du.abs()) @ Wu.double().abs()
        _check("dX", dX.t, ref, e + _store(kind, ref.abs() + e))
    for c, out, d, r in (("g", dWg, dg, rg), ("u", dWu, du, ru)):
        if c in want:
            ref = d.T @ X.double()
            e = (r + (M + 2) * U * d.abs()).T @ X.double().abs()
            _check("dW" + c, out.t, ref, e + _store(kind, ref.abs() + e))
    for c, out, d, e in (("b", dbg, dg, eg), ("c", dbu, du, eu)):
        if c in want:
            _check("db", out[:N], d.sum(0), e.sum(0) + (M + 2) * U * d.abs().sum(0) + TINY["f32"])
        assert bool(out[N].isnan())
    for m, c in ((dX, "x"), (dWg, "g"), (dWu, "u")):
        assert m.others_untouched() if c in want else bool(m.flat.isnan().all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES + LARGE, ids=str)
def test_glu_backward(torch, igc, ws, size, kind):
    i = (SIZES + LARGE).index(size)
    for j, want in enumerate(("xgubc", "xgu", "x", "g", "uc", "b")):
        if j > 1 and size in LARGE:
            break
        _glu_backward(torch, igc, ws, size, kind, ACTS[(i + j) % 6], want, seed=i)


# Outputs (rows, columns) and reductions that take each tile, whole, in splits,
# and with the last round of tiles in splits.
PRODUCTS = [(136, 10960, 72), (72, 4280, 3520), (4632, 1696, 840), (912, 12344, 336), (392, 8208, 3336), (1440, 11224, 1384), (72, 208, 1448),
            (72, 208, 3384), (544, 13128, 1128), (520, 512, 8192), (104, 2048, 520), (520, 4096, 1024)]
PRODUCTS_GLU = [(72, 2384, 3424), (280, 11312, 1176), (424, 12488, 408), (136, 2704, 14288), (1464, 5464, 1296), (72, 8208, 2456), (72, 208, 840),
                (72, 208, 1864), (72, 1400, 9120), (280, 11008, 1456), (72, 7176, 72), (136, 2904, 14288)]
# Rows that the direct loads do not take: odd lengths, and a start off the 16 bytes.
UNALIGNED = [(200, 1000, 2049, 0, 0), (727, 1345, 1531, 0, 0), (300, 1001, 2001, 2, 1), (1000, 1500, 1500, 0, 4), (520, 2000, 1000, 8, 1),
             (96, 999, 1601, 0, 0), (2100, 1300, 260, 0, 2), (70, 2049, 2047, 3, 0)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", PRODUCTS, ids=str)
def test_linear_products(torch, igc, ws, size, kind):
    m, n, r = size
    _linear_forward(torch, igc, ws, (m, n, r, 0, 0), kind, "silu", True, True, True, "f32" if kind == "f16" else kind)
    _linear_backward(torch, igc, ws, (m, r, n, 0, 0), kind, "relu", "x")
    _linear_backward(torch, igc, ws, (r, m, n, 0, 0), kind, "none", "w")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", PRODUCTS_GLU, ids=str)
def test_glu_products(torch, igc, ws, size, kind):
    m, n, r = size
    _glu(torch, igc, ws, (m, n, r, 0, 0), kind, "silu", True, True)


@pytest.mark.parametrize("size", [(520, 4104, 1024), (632, 4096, 2432), (1000, 8192, 1000), (40, 8192, 1024), (4104, 520, 1032)], ids=str)
def test_both_products_of_a_layer(torch, igc, ws, size):
    _linear_backward(torch, igc, ws, size + (0, 0), "bf16", "gelu", "xwb")
    _linear_backward(torch, igc, ws, size + (0, 0), "f16", "none", "xw")
    _glu_backward(torch, igc, ws, size + (0, 0), "f16", "silu", "xgub")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", UNALIGNED, ids=str)
def test_rows_that_are_padded(torch, igc, ws, size, kind):
    _linear_forward(torch, igc, ws, size, kind, "gelu", True, True, True, "f32")
    _glu(torch, igc, ws, size, kind, "silu", True, True)
    _linear_backward(torch, igc, ws, size, kind, "none", "xw")
    _linear_backward(torch, igc, ws, size, kind, "none", "x")
    _linear_backward(torch, igc, ws, size, kind, "silu", "xwb")
    _glu_backward(torch, igc, ws, size, kind, "silu", "xgubc")
    _glu_backward(torch, igc, ws, size, kind, "gelu", "u")


def test_empty_batch_sets_weight_gradients_to_zero(torch, igc, ws):
    dW, db = torch.full((24, 16), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((24,), float("nan"), device="cuda")
    igc.linear_backward(0, 24, 16, None, 24, Z=None, ldz=24, X=None, ldx=16, dW=dW, lddw=16, dbias=db, act=igc.IGC_ACT_SILU, workspace=ws)
    assert int(dW.count_nonzero()) == 0 and int(db.count_nonzero()) == 0
    dWg, dWu = torch.full_like(dW, float("nan")), torch.full_like(dW, float("nan"))
    igc.glu_backward(0, 24, 16, None, 24, None, 24, None, 24, X=None, ldx=16, dWg=dWg, lddwg=16, dWu=dWu, lddwu=16, workspace=ws)
    assert int(dWg.count_nonzero()) == 0 and int(dWu.count_nonzero()) == 0
    dX = torch.full((8, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    igc.linear_backward(8, 0, 16, None, 0, W=None, ldw=16, dX=dX, lddx=16, workspace=ws)
    assert int(dX.count_nonzero()) == 0


def test_extreme_activations(torch, igc, ws):
    """Sums far out in both tails, infinities and NaN go where the formulas send them."""
    vals = torch.tensor([-1e30, -300.0, -80.0, -12.0, -5.5, -0.0, 0.0, 1e-30, 5.5, 12.0, 80.0, 300.0, 1e30, float("inf"), float("nan"), -3.0],
                        device="cuda")
    one = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(16, 8, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(1, 16, device="cuda")
    for act in ACTS:
        igc.linear_forward(1, 16, 8, one, 8, zero, 8, Y, 16, y_type=igc.IGC_F32, bias=vals, act=_act_id(igc, act), workspace=ws)
        ref = _f(act, vals.double())[0]
        got = Y[0].double()
        assert bool(got[14].isnan()), act
        fin = torch.isfinite(ref)
        assert bool((torch.isfinite(got) | ~fin).all()), (act, got, ref)
        assert float(((got - ref).abs() - 8 * U * (vals.double().abs() + 1)).nan_to_num(-1)[fin].max()) <= 0, (act, got, ref)
        assert got[13] == ref[13] or act == "gelu_tanh", act


def test_gradients_against_differences(torch, igc, ws):
    """dX, dW and db of a sum of outputs agree with central differences of the forward pass in 64 bits."""
    M, N, K = 6, 10, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    X, Wg, Wu = (torch.randn(r, K, generator=gen, device="cuda").bfloat16() for r in (M, N, N))
    bg, bu = (torch.randn(N, generator=gen, device="cuda") for _ in range(2))
    c = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    H, G, Uo = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    igc.glu_forward(M, N, K, X, K, Wg, K, Wu, K, H, N, bias_g=bg, bias_u=bu, G=G, ldg=N, U=Uo, ldu=N, workspace=ws)
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    db1, db2 = torch.empty_like(bg), torch.empty_like(bu)
    igc.glu_backward(M, N, K, c, N, G, N, Uo, N, X=X, ldx=K, Wg=Wg, ldwg=K, Wu=Wu, ldwu=K, dX=dX, lddx=K, dWg=dWg, lddwg=K,
                     dWu=dWu, lddwu=K, dbias_g=db1, dbias_u=db2, workspace=ws)

    def loss(v):
        g, u = v[0] @ v[1].T + v[3], v[0] @ v[2].T + v[4]
        return float((g * torch.sigmoid(g) * u * c.double()).sum())

    v = [t.double() for t in (X, Wg, Wu, bg, bu)]
    rng = np.random.default_rng(3)
    # G and U are kept in bf16 and D is rounded to it: each term within 3 half
    # steps through slopes of at most ~2.5; 2% of the largest gradient covers
    # the sums of 10 to 16 such terms
    for t, got in zip(v, (dX, dWg, dWu, db1, db2)):
        scale = float(got.double().abs().max())
        for _ in range(6):
            i = tuple(int(rng.integers(0, n)) for n in t.shape)
            keep = float(t[i])
            t[i] = keep + 1e-4
            up = loss(v)
            t[i] = keep - 1e-4
            down = loss(v)
            t[i] = keep
            assert abs((up - down) / 2e-4 - float(got[i])) <= 0.02 * scale


def test_split_reduction_is_deterministic(torch, igc, ws):
    first = _linear_forward(torch, igc, ws, (40, 64, 8192, 0, 0), "bf16", "silu", True, False, False, "f32")
    for _ in range(4):
        again = _linear_forward(torch, igc, ws, (40, 64, 8192, 0, 0), "bf16", "silu", True, False, False, "f32")
        assert torch.equal(first, again)


def test_another_stream_and_its_own_workspace(torch, igc, ws):
    s = torch.cuda.Stream()
    own = torch.full_like(ws, 255)
    torch.cuda.synchronize()
    _linear_forward(torch, igc, own, (130, 200, 4096, 0, 0), "f16", "gelu", True, True, True, "f16", stream=s)


def test_graph_replays(torch, igc):
    """A captured step (gated block, projection, both backward passes, clipping) gives the eager results on every replay."""
    M, N, K = 96, 328, 256
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    X, W1, W2, W3 = (torch.randn(r, c, generator=gen, device="cuda").bfloat16() * 0.06 for r, c in ((M, K), (N, K), (N, K), (K, N)))
    dY = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    H, G, Uo, Y, dH, dX = new(M, N), new(M, N), new(M, N), new(M, K), new(M, N), new(M, K)
    d1, d2, d3, db, norm = new(N, K), new(N, K), new(K, N), torch.empty(K, device="cuda"), torch.empty(1, device="cuda")
    clipped = [torch.empty_like(t) for t in (d1, d2, d3)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step():
        igc.glu_forward(M, N, K, X, K, W1, K, W2, K, H, N, G=G, ldg=N, U=Uo, ldu=N, workspace=ws)
        igc.linear_forward(M, K, N, H, N, W3, N, Y, K, R=X, ldr=K, workspace=ws)
        igc.linear_backward(M, K, N, dY, K, X=H, ldx=N, W=W3, ldw=N, dX=dH, lddx=N, dW=d3, lddw=N, dbias=db, workspace=ws)
        igc.glu_backward(M, N, K, dH, N, G, N, Uo, N, X=X, ldx=K, Wg=W1, ldwg=K, Wu=W2, ldwu=K, dX=dX, lddx=K, dWg=d1, lddwg=K,
                         dWu=d2, lddwu=K, workspace=ws)
        igc.grad_clip([d1, d2, d3], 0.5, norm, out=clipped, workspace=ws)

    outs = [H, Y, dX, db, norm, *clipped]
    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, e in zip(outs, eager):
            assert torch.equal(t, e)
        step()
        torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# Clipping
# ---------------------------------------------------------------------------
def _clip(torch, igc, ws, sizes, kinds, share, in_place=False, shift=0, scale=0.1):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(77)
    grads = []
    for n, k in zip(sizes, kinds):
        flat = torch.full((n + shift + 8,), float("nan"), dtype=_dt(torch, k), device="cuda")
        flat[shift:shift + n] = torch.randn(n, generator=gen, device="cuda") * scale
        grads.append(flat[shift:shift + n])
    total = math.sqrt(sum(float(torch.dot(g.double(), g.double())) for g in grads))
    limit = float(np.float32(share * total))
    before = [g.double().clone() for g in grads]
    outs = grads if in_place else [torch.full((n + shift + 8,), float("nan"), dtype=g.dtype, device="cuda")[shift:shift + n]
                                   for n, g in zip(sizes, grads)]
    norm = torch.full((1,), float("nan"), device="cuda")
    assert igc.grad_clip_workspace_size(grads, limit, norm) <= ws.numel()
    igc.grad_clip(grads, limit, norm, out=None if in_place else outs, workspace=ws)
    torch.cuda.synchronize()
    # the norm: one rounding to fp32 of a sum in 64 bits
    assert abs(float(norm) - total) <= 2 * U * total
    factor = min(1.0, limit / (total + 1e-6))
    for b, o, k in zip(before, outs, kinds):
        ref = b * factor
        # the factor and the product round once each in fp32, the store once
        _check("out", o, ref, 4 * U * ref.abs() + _store(k, ref.abs()))
        if factor == 1.0:
            assert torch.equal(o.double(), b)
    return norm


@pytest.mark.parametrize("share", [0.0, 0.3, 2.0])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_clip_mixed(torch, igc, ws, share, in_place, shift):
    sizes = [1, 2, 3, 7, 8, 9, 0, 255, 4096, 8191, 8192, 8193, 70001, 0]
    _clip(torch, igc, ws, sizes, [("f16", "bf16", "f32")[i % 3] for i in range(len(sizes))], share, in_place, shift)


@pytest.mark.parametrize("count", [1, 63, 64, 65, 200])
def test_clip_many_tensors(torch, igc, ws, count):
    sizes = [1 + (i * 977) % 5000 for i in range(count)]
    _clip(torch, igc, ws, sizes, [("bf16", "f32", "f16")[i % 3] for i in range(count)], 0.5)


def test_clip_large(torch, igc, ws):
    _clip(torch, igc, ws, [1 << 24, 12345677, 3], ["bf16", "f32", "f16"], 0.1)


def test_clip_nothing_and_no_tensors(torch, igc, ws):
    norm = torch.full((1,), float("nan"), device="cuda")
    igc.grad_clip([], 1.0, norm, workspace=ws)
    assert float(norm) == 0.0
    z = torch.zeros(100, device="cuda")
    igc.grad_clip([z], 1.0, norm, workspace=ws)
    assert float(norm) == 0.0 and int(z.count_nonzero()) == 0


def test_clip_values_whose_squares_leave_fp32(torch, igc, ws):
    g = torch.full((1000,), 1e25, dtype=torch.bfloat16, device="cuda")
    norm = torch.empty(1, device="cuda")
    value = float(g[0].double())
    igc.grad_clip([g], 1.0, norm, workspace=ws)
    assert abs(float(norm) / (value * math.sqrt(1000)) - 1) <= 2 * U
    assert abs(float(g[0]) * math.sqrt(1000) - 1) <= HALF["bf16"] * 1.01 + 4 * U
    small = torch.full((1000,), 1e-30, device="cuda")
    igc.grad_clip([small], 1.0, norm, workspace=ws)
    assert abs(float(norm) / (float(torch.tensor(1e-30, dtype=torch.float32)) * math.sqrt(1000)) - 1) <= 2 * U


def test_clip_not_finite(torch, igc, ws):
    norm = torch.empty(1, device="cuda")
    g = torch.ones(5000, device="cuda")
    g[4321] = float("nan")
    igc.grad_clip([g], 1.0, norm, workspace=ws)
    assert bool(norm.isnan()) and bool(g.isnan().all())
    g = torch.ones(5000, device="cuda")
    g[17] = float("-inf")
    igc.grad_clip([g], 1.0, norm, workspace=ws)
    assert bool(norm.isinf()) and bool(g[17].isnan()) and int(g.nan_to_num(0.0).count_nonzero()) == 0


def test_offsets_past_32_bits(torch, igc, ws):
    """Rows that start more than 2^32 bytes into their matrices: the tiles (70000 rows of a leading dimension of 40000), the
    streaming kernel and the copies into padded rows (a few rows, 2^30 apart)."""
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    M, N, K, ld = 70000, 96, 128, 40000
    big = lambda cols: torch.empty(M, ld, dtype=torch.float16, device="cuda")[:, :cols]  # noqa: E731
    X, Y, Z, dY, dX = big(K), big(N), big(N), big(N), big(K)
    X.copy_(torch.randn(M, K, generator=gen, device="cuda"))
    dY.copy_(torch.randn(M, N, generator=gen, device="cuda"))
    W = (torch.randn(N, K, generator=gen, device="cuda") * K ** -0.5).half()
    igc.linear_forward(M, N, K, X, ld, W, K, Y, ld, type=igc.IGC_F16, act=igc.IGC_ACT_SILU, Z=Z, ldz=ld, workspace=ws)
    dW, db = torch.empty_like(W), torch.empty(N, device="cuda")
    igc.linear_backward(M, N, K, dY, ld, Z=Z, ldz=ld, X=X, ldx=ld, W=W, ldw=K, dX=dX, lddx=ld, dW=dW, lddw=K, dbias=db,
                        type=igc.IGC_F16, act=igc.IGC_ACT_SILU, workspace=ws)
    rows = slice(M - 3000, M)
    x, w = X[rows].double(), W.double()
    z, s = x @ w.T, x.abs() @ w.abs().T
    ez = (K + 2) * U * s
    _check("Z", Z[rows], z, ez + _store("f16", z.abs() + ez))
    f = _f("silu", z)[0]
    _check("Y", Y[rows], f, 1.13 * ez + 8 * U * (z.abs() + 1) + _store("f16", f.abs() + ez))
    d = dY.double() * _f("silu", Z.double())[1]
    ed = 8 * U * dY.double().abs() * (1 + Z.double().abs())
    er = ed + _store("f16", d.abs() + ed)
    e = er[rows] @ w.abs() + (N + 2) * U * (d[rows].abs() @ w.abs())
    _check("dX", dX[rows], d[rows] @ w, e + _store("f16", (d[rows] @ w).abs() + e))
    ref = d.T @ X.double()
    e = (er + (M + 2) * U * d.abs()).T @ X.double().abs()
    _check("dW", dW, ref, e + _store("f16", ref.abs() + e))
    _check("db", db, d.sum(0), ed.sum(0) + (M + 2) * U * d.abs().sum(0) + TINY["f32"])
    del X, Y, Z, dY, dX, d, ed, er
    torch.cuda.empty_cache()
    far = 1 << 30
    for rows, cols, outs in ((3, 521, 40), (70, 1200, 300)):  # the streaming kernel; padded or any rows
        if rows * far * 2 > 16 << 30:
            far = (8 << 30) // rows // 2 * 2 + 1  # elements: 16 GiB in all, odd rows
        flat = torch.empty(rows * far, dtype=torch.bfloat16, device="cuda")
        X = flat.view(rows, far)[:, :cols]
        X.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))
        W = (torch.randn(outs, cols, generator=gen, device="cuda") * cols ** -0.5).bfloat16()
        Y = torch.empty(rows, outs, device="cuda")
        igc.linear_forward(rows, outs, cols, X, far, W, cols, Y, outs, y_type=igc.IGC_F32, workspace=ws)
        ref, s = X.double() @ W.double().T, X.double().abs() @ W.double().abs().T
        _check("Y", Y, ref, (cols + 4) * U * s + 8 * U * (ref.abs() + 1) + _store("f32", ref.abs()))
        del flat, X
        torch.cuda.empty_cache()
