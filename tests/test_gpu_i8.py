"""Products in 8 bits on the GPU: whole sums to the bit, everything after them
against the formula in 64 bits.

Tolerances, from the arithmetic (u = 2^-24): the sum's conversion, two scales and
the bias are a rounding each: 4 u |z - b| + u |z|; the activations as for the 16-bit
products (8 u of what they are applied to, a slope of at most 1.13); a store by half
a step of its type.
"""
from __future__ import annotations

import pytest

from test_gpu_ffn import ACTS, Mat, U, _act_id, _check, _f, _store, _type, igc, torch, ws  # noqa: F401

pytestmark = pytest.mark.gpu


class Ints:
    """rows x cols of int8 in rows of a longer buffer of other values, `shift` bytes off the allocation's start."""

    def __init__(self, torch, rows, cols, ld, shift, gen, low=-127, high=127):  # noqa: F811
        self.ld, self.rows, self.cols = ld, rows, cols
        self.flat = torch.randint(-128, 128, (shift + rows * ld + 64,), generator=gen, device="cuda", dtype=torch.int8)
        self.t = torch.as_strided(self.flat, (rows, cols), (ld, 1), shift)
        self.ptr = self.flat.data_ptr() + shift
        if rows and cols:
            self.t.copy_(torch.randint(low, high + 1, (rows, cols), generator=gen, device="cuda", dtype=torch.int8))


# (M, N, K, extra row length of the operands, shift in bytes): few rows and many, tiles' ends, every alignment
SIZES = [
    (1, 1, 1, 0, 0), (1, 16, 16, 0, 0), (3, 5, 7, 2, 1), (1, 300, 1040, 0, 0), (2, 1001, 333, 0, 3), (5, 64, 0, 3, 0), (70, 64, 0, 8, 0),
    (16, 96, 2048, 0, 0), (17, 33, 65, 0, 0), (24, 520, 1000, 8, 8), (24, 520, 1000, 4, 4), (33, 130, 272, 0, 0), (63, 200, 144, 16, 16),
    (64, 64, 128, 0, 0), (65, 257, 129, 1, 3), (70, 40, 13, 0, 0), (128, 256, 512, 0, 0), (131, 1000, 520, 0, 0), (200, 264, 336, 16, 32),
    (256, 512, 256, 0, 0), (300, 777, 1001, 0, 0), (513, 640, 192, 0, 0), (48, 4096, 4096, 0, 0), (1, 10944, 2048, 0, 0),
]
LARGE = [(2100, 2056, 528, 0, 0), (1025, 4104, 400, 16, 0), (4100, 1030, 272, 0, 2), (3400, 4104, 272, 0, 0), (3400, 144, 8208, 16, 16),
         (144, 3400, 8208, 0, 0), (520, 4104, 8192, 0, 0), (1, 4096, 131071, 0, 0), (100, 200, 131056, 0, 0)]


def _scales(torch, gen, M, N):  # noqa: F811
    return torch.rand(M, generator=gen, device="cuda") * 0.05 + 1e-4, torch.rand(N, generator=gen, device="cuda") * 2e-3 + 1e-5


def _sums(x, w):
    return x.double() @ w.double().T  # (whole numbers below 2^53)


def _z(acc, s, w, b):
    z = acc * s.double()[:, None] * w.double()[None, :]
    e = 4 * U * z.abs()
    if b is not None:
        z = z + b.double()
    return z, e + U * z.abs()


def _linear(torch, igc, ws, size, act, y, bias, residual, seed=0, stream=None):  # noqa: F811
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5000 + seed)
    X, W = Ints(torch, M, K, K + more, shift, gen), Ints(torch, N, K, K + more, shift, gen, -128)
    xs, wscale = _scales(torch, gen, M, N)
    b = torch.randn(N, generator=gen, device="cuda") if bias else None
    R = Mat(torch, M, N, y, N + more, shift, gen) if residual else None
    Y = Mat(torch, M, N, y, N + more, shift)
    kw = dict(y_type=_type(igc, y), act=_act_id(igc, act), bias=b, R=R and R.ptr, ldr=N + more)
    args = (M, N, K, X.ptr, X.ld, xs, W.ptr, W.ld, wscale, Y.ptr, Y.ld)
    need = igc.linear_i8_workspace_size(*args, **kw)
    assert need <= ws.numel()
    ws[need:need + 256] = 255
    igc.linear_i8(*args, **kw, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert bool((ws[need:need + 256] == 255).all())
    z, ez = _z(_sums(X.t, W.t), xs, wscale, b)
    f = _f(act, z)[0]
    ref = f + R.double() if residual else f
    ey = 1.13 * ez + 8 * U * (z.abs() + f.abs() + ref.abs() + 1)
    _check("Y", Y.t, ref, ey + _store(y, ref.abs() + ey))
    assert Y.others_untouched()
    first = Y.t.clone()
    igc.linear_i8(*args, **kw, workspace=ws, stream=stream)
    assert torch.equal(Y.t, first)


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_i8(torch, igc, ws, size):  # noqa: F811
    i = SIZES.index(size)
    for j in range(4):
        n = i + 7 * j
        _linear(torch, igc, ws, size, ACTS[n % 6], ("f16", "bf16", "f32")[n % 3], n % 2 == 0, n % 3 != 1, seed=n)


@pytest.mark.parametrize("y", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("size", LARGE, ids=str)
def test_linear_i8_large(torch, igc, ws, size, y):  # noqa: F811
    _linear(torch, igc, ws, size, "gelu", y, True, True)


@pytest.mark.parametrize("size", [(1, 64, 4096, 0, 0), (40, 100, 4096, 0, 0), (300, 300, 4096, 0, 0), (300, 300, 4000, 0, 1), (30, 70, 131071, 0, 0),
                                  (200, 70, 131071, 0, 0), (256, 256, 16384, 0, 0)], ids=str)
def test_sums_are_exact(torch, igc, ws, size):  # noqa: F811
    """Without scales in the way: every sum, converted to fp32, to the bit; also at the largest sums that K allows."""
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    one, ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    for low, high in ((-128, 127), (-128, -128), (127, 127)):
        X, W = Ints(torch, M, K, K + more, shift, gen, low, high), Ints(torch, N, K, K + more, shift, gen, low, high)
        Y = torch.empty(M, N, device="cuda")
        igc.linear_i8(M, N, K, X.ptr, X.ld, one, W.ptr, W.ld, ones, Y, N, y_type=igc.IGC_F32, workspace=ws)
        assert torch.equal(Y, _sums(X.t, W.t).float())


def _glu(torch, igc, ws, size, act, kind, bias, seed=0):  # noqa: F811
    M, N, K, more, shift = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6000 + seed)
    X, Wg, Wu = (Ints(torch, r, K, K + more, shift, gen) for r in (M, N, N))
    xs, sg = _scales(torch, gen, M, N)
    su = sg.flip(0).contiguous()
    bg, bu = (torch.randn(N, generator=gen, device="cuda") if bias else None for _ in range(2))
    if seed % 3 == 2:
        bg = None
    H = Mat(torch, M, N, kind, N + more, shift)
    kw = dict(type=_type(igc, kind), act=_act_id(igc, act), bias_g=bg, bias_u=bu)
    args = (M, N, K, X.ptr, X.ld, xs, Wg.ptr, Wg.ld, sg, Wu.ptr, Wu.ld, su, H.ptr, H.ld)
    need = igc.glu_i8_workspace_size(*args, **kw)
    assert need <= ws.numel()
    ws[need:need + 256] = 255
    igc.glu_i8(*args, **kw, workspace=ws)
    torch.cuda.synchronize()
    assert bool((ws[need:need + 256] == 255).all())
    g, eg = _z(_sums(X.t, Wg.t), xs, sg, bg)
    u, eu = _z(_sums(X.t, Wu.t), xs, su, bu)
    f = _f(act, g)[0]
    ref = f * u
    eh = (1.13 * eg + 8 * U * (g.abs() + f.abs() + 1)) * (u.abs() + eu) + f.abs() * eu + 2 * U * ref.abs()
    _check("H", H.t, ref, eh + _store(kind, ref.abs() + eh))
    assert H.others_untouched()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_glu_i8(torch, igc, ws, size, kind):  # noqa: F811
    i = SIZES.index(size)
    for j in range(2):
        _glu(torch, igc, ws, size, ACTS[(i + 3 * j) % 6], kind, j == 0, seed=i + j)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", LARGE[:7], ids=str)
def test_glu_i8_large(torch, igc, ws, size, kind):  # noqa: F811
    _glu(torch, igc, ws, size, "silu", kind, True)


@pytest.mark.parametrize("M", [1, 40, 200])
def test_operands_of_different_alignment(torch, igc, ws, M):  # noqa: F811
    """Only one of the operands can be loaded as it is."""
    N, K = 300, 640
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for x_more, x_shift, w_more, w_shift in ((0, 0, 1, 0), (3, 0, 0, 0), (0, 1, 0, 0), (16, 16, 0, 5), (4, 4, 16, 0)):
        X, W = Ints(torch, M, K, K + x_more, x_shift, gen), Ints(torch, N, K, K + w_more, w_shift, gen)
        V = Ints(torch, N, K, K, 0, gen)
        xs, wscale = _scales(torch, gen, M, N)
        Y, H = torch.empty(M, N, device="cuda"), torch.empty(M, N, dtype=torch.float16, device="cuda")
        igc.linear_i8(M, N, K, X.ptr, X.ld, xs, W.ptr, W.ld, wscale, Y, N, y_type=igc.IGC_F32, workspace=ws)
        z, ez = _z(_sums(X.t, W.t), xs, wscale, None)
        _check("Y", Y, z, ez)
        igc.glu_i8(M, N, K, X.ptr, X.ld, xs, W.ptr, W.ld, wscale, V.ptr, V.ld, wscale, H, N, type=igc.IGC_F16, act=igc.IGC_ACT_RELU, workspace=ws)
        u, eu = _z(_sums(X.t, V.t), xs, wscale, None)
        ref = z.clamp(min=0) * u
        eh = 1.1 * (ez * u.abs() + eu * z.abs()) + 8 * U * (z.abs() + 1) * u.abs() + 2 * U * ref.abs()
        _check("H", H, ref, eh + _store("f16", ref.abs() + eh))


def test_rows_that_are_not_finite_and_rows_of_zeros(torch, igc, ws):  # noqa: F811
    """quantize_rows' scales carry through: NaN rows are NaN in Y, zero rows leave act(bias) + R, the others are as without them."""
    for M in (5, 130):
        N, K = 96, 512
        gen = torch.Generator(device="cuda")
        gen.manual_seed(2)
        x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
        x[1] = 0
        x[2, 5], x[M - 1, K - 1] = float("nan"), float("inf")
        Q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        igc.quantize_rows(M, K, x, K, Q, K, s)
        W = Ints(torch, N, K, K, 0, gen)
        wscale, b = torch.rand(N, generator=gen, device="cuda"), torch.randn(N, generator=gen, device="cuda")
        R = torch.randn(M, N, generator=gen, device="cuda")
        Y = torch.empty(M, N, device="cuda")
        igc.linear_i8(M, N, K, Q, K, s, W.ptr, K, wscale, Y, N, y_type=igc.IGC_F32, bias=b, R=R, ldr=N, workspace=ws)
        bad = torch.zeros(M, dtype=torch.bool, device="cuda")
        bad[2] = bad[M - 1] = True
        assert bool(Y[bad].isnan().all()) and not bool(Y[~bad].isnan().any())
        assert torch.equal(Y[1], b + R[1])


def test_bounds_of_the_outputs(torch, igc, ws):  # noqa: F811
    """Sums times scales past fp16's range are infinities of their sign."""
    M, N, K = 40, 64, 256
    X, W = torch.full((M, K), 127, dtype=torch.int8, device="cuda"), torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    W[::2] = -127
    s = torch.full((M,), 3.0, device="cuda")
    Y = torch.empty(M, N, dtype=torch.float16, device="cuda")
    igc.linear_i8(M, N, K, X, K, s, W, K, torch.ones(N, device="cuda"), Y, N, y_type=igc.IGC_F16, workspace=ws)
    assert bool((Y[:, ::2] == float("-inf")).all()) and bool((Y[:, 1::2] == float("inf")).all())


def test_weights_past_32_bit_offsets(torch, igc, ws):  # noqa: F811
    """Weight rows that begin more than 2^32 bytes into their matrix, few and many rows of X."""
    N, K, ld = 300, 256, 1 << 24
    flat = torch.empty((N - 1) * ld + K, dtype=torch.int8, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    w = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    torch.as_strided(flat, (N, K), (ld, 1)).copy_(w)
    for M in (3, 100):
        x = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
        xs, wscale = _scales(torch, gen, M, N)
        Y, want = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        igc.linear_i8(M, N, K, x, K, xs, flat, ld, wscale, Y, N, y_type=igc.IGC_F32, workspace=ws)
        igc.linear_i8(M, N, K, x, K, xs, w, K, wscale, want, N, y_type=igc.IGC_F32, workspace=ws)
        assert torch.equal(Y, want)


def test_no_rows_or_columns(torch, igc):  # noqa: F811
    y = torch.full((8,), 7.0, device="cuda")
    igc.linear_i8(0, 4, 4, None, 4, None, y, 4, y, y, 4, y_type=igc.IGC_F32)
    igc.linear_i8(4, 0, 4, y, 4, y, None, 4, None, y, 0, y_type=igc.IGC_F32)
    igc.glu_i8(0, 4, 4, None, 4, None, y, 4, y, y, 4, y, y, 4)
    assert igc.linear_i8_workspace_size(0, 4, 4, None, 4, None, y, 4, y, y, 4) == 0
    assert bool((y == 7).all())
