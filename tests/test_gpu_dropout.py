"""Dropout on the GPU: bit for bit the formula, with the generator's words from
the tests' own implementation (tests/philox.py)."""
from __future__ import annotations

import numpy as np
import pytest

from philox import border, words
from test_gpu_ffn import Mat, _dt, _type, igc, torch  # noqa: F401

pytestmark = pytest.mark.gpu

SEED = 0x0123456789ABCDEF


def _want(torch, x, r, y_kind, p, seed, offset):  # noqa: F811
    """fp32 product and sum, each rounded once, then the type: what the formula is in those operations."""
    T = border(p)
    keep = torch.from_numpy(words(x.shape[0], x.shape[1], seed, offset) >= T).cuda()
    scale = torch.tensor(0.0 if T == 2 ** 32 else 2.0 ** 32 / (2 ** 32 - T), dtype=torch.float32, device="cuda")
    y = torch.where(keep, x.float() * scale, torch.zeros((), device="cuda"))
    if r is not None:
        y = y + r.float()
    return y.to(_dt(torch, y_kind)), keep


# (M, N, extra row length, shift)
SIZES = [(1, 1, 0, 0), (1, 4, 0, 0), (3, 5, 1, 1), (2, 8, 0, 0), (7, 9, 0, 0), (1, 4096, 0, 0), (64, 64, 8, 8), (33, 1001, 0, 0), (300, 520, 8, 0),
         (5, 20003, 2, 3), (3000, 7, 0, 0), (1111, 1200, 0, 0), (2100, 4096, 0, 0)]
TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"), ("f32", "f16"), ("bf16", "f32"), ("f32", "bf16")]


@pytest.mark.parametrize("x_kind,y_kind", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_dropout(torch, igc, size, x_kind, y_kind):  # noqa: F811
    M, N, more, shift = size
    i = SIZES.index(size)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(i)
    X = Mat(torch, M, N, x_kind, N + more, shift, gen)
    R = Mat(torch, M, N, y_kind, N + more, shift, gen)
    step = torch.tensor([2 ** 33 + 5], dtype=torch.int64, device="cuda")
    for p, residual, offset, stepped in ((0.1, True, 0, False), (0.5, False, 2 ** 32 - 3, True), (1 / 3, True, 2 ** 64 - 1, True)):
        Y = Mat(torch, M, N, y_kind, N + more, shift)
        igc.dropout(M, N, X.ptr, X.ld, Y.ptr, Y.ld, p, SEED + i, offset, step=step if stepped else None, R=R.ptr if residual else None, ldr=R.ld,
                    type=_type(igc, x_kind), y_type=_type(igc, y_kind))
        torch.cuda.synchronize()
        want, _ = _want(torch, X.t, R.t if residual else None, y_kind, p, SEED + i, (offset + (2 ** 33 + 5 if stepped else 0)) % 2 ** 64)
        assert torch.equal(Y.t, want)
        assert Y.others_untouched()


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
def test_ends_of_p_and_values_that_are_not_finite(torch, igc, kind):  # noqa: F811
    M, N = 37, 203
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(M, N, generator=gen, device="cuda").to(_dt(torch, kind))
    x[::3, ::5], x[1::3, ::7], x[2::3, ::4] = float("inf"), float("nan"), float("-inf")
    r = torch.randn(M, N, generator=gen, device="cuda").to(_dt(torch, kind))
    for p in (0.0, 2.0 ** -34, 2.0 ** -32, 0.9, 1 - 2.0 ** -32, 1 - 2.0 ** -34, 1.0):
        for res in (None, r):
            y = torch.empty_like(x)
            igc.dropout(M, N, x, N, y, N, p, 9, R=res, ldr=N, type=_type(igc, kind))
            want, keep = _want(torch, x, res, kind, p, 9, 0)
            assert torch.equal(y.nan_to_num(123.0), want.nan_to_num(123.0)) and torch.equal(y.isnan(), want.isnan())
            if p in (0.0, 2.0 ** -34):
                assert bool(keep.all())
            if p in (1.0, 1 - 2.0 ** -34):
                assert not bool(keep.any()) and torch.equal(y, torch.zeros_like(x) if res is None else r)


def test_in_place_and_backward(torch, igc):  # noqa: F811
    """Y on X or on R; the same call on dY is the gradient, by differences too."""
    M, N, p, seed, offset = 50, 333, 0.3, 77, 6
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x, r, dy = (torch.randn(M, N, generator=gen, device="cuda") for _ in range(3))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    kw = dict(type=igc.IGC_F32)
    igc.dropout(M, N, x, N, y, N, p, seed, offset, R=r, ldr=N, **kw)
    on_x, on_r = x.clone(), r.clone()
    igc.dropout(M, N, on_x, N, on_x, N, p, seed, offset, R=r, ldr=N, **kw)
    igc.dropout(M, N, x, N, on_r, N, p, seed, offset, R=on_r, ldr=N, **kw)
    assert torch.equal(on_x, y) and torch.equal(on_r, y)
    igc.dropout(M, N, dy, N, dx, N, p, seed, offset, **kw)
    # y is linear in x, element by element: a step of 1 in x moves y by 1 / (1 - p) or not at all, up to the rounding of y
    y1 = torch.empty_like(x)
    igc.dropout(M, N, x + 1, N, y1, N, p, seed, offset, R=r, ldr=N, **kw)
    slope = (y1.double() - y.double())
    assert float((dx.double() - dy.double() * slope).abs().max()) <= 16 * 2.0 ** -24 * float((dy.abs() * (x.abs() + r.abs() + 2)).max())
    assert 0.25 < float((dx == 0).double().mean()) < 0.35


def test_mask_does_not_depend_on_layout(torch, igc):  # noqa: F811
    """Leading dimensions, types and the rest of the matrix leave the mask as it is; seed, offset and step change it."""
    M, N = 20, 130
    ones = torch.ones(M, N, device="cuda")
    masks = []
    for seed, offset, step in ((3, 4, None), (3, 0, 4), (4, 4, None), (3, 5, None), (3 + 2 ** 32, 4, None), (3, 4 + 2 ** 32, None)):
        y = torch.empty_like(ones)
        s = None if step is None else torch.tensor([step], device="cuda")
        igc.dropout(M, N, ones, N, y, N, 0.5, seed, offset, step=s, type=igc.IGC_F32)
        masks.append(y != 0)
    assert torch.equal(masks[0], masks[1])
    for i in range(2, 6):
        for j in range(i):
            if j != 1:
                # two independent masks agree on half of the 2600 elements; six deviations of 25
                assert abs(float((masks[i] == masks[j]).double().mean()) - 0.5) < 0.06, (i, j)
    wide, out = torch.ones(M, N + 9, device="cuda").bfloat16(), torch.zeros(M, N + 3, device="cuda")
    igc.dropout(M, N, wide, N + 9, out, N + 3, 0.5, 3, 4, type=igc.IGC_BF16, y_type=igc.IGC_F32)
    assert torch.equal(out[:, :N] != 0, masks[0]) and not bool(out[:, N:].any())
    top = torch.empty(7, 60, device="cuda")
    igc.dropout(7, 60, ones, N, top, 60, 0.5, 3, 4, type=igc.IGC_F32)
    assert torch.equal(top != 0, masks[0][:7, :60])


def test_captured_calls_follow_the_step(torch, igc):  # noqa: F811
    """A replay reads the number again; forward and backward of one replay agree; eager calls between replays change nothing."""
    M, N = 65, 515
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    igc.dropout(M, N, x, N, y, N, 0.2, 8, 1, step=step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        igc.dropout(M, N, x, N, y, N, 0.2, 8, 1, step=step)
        igc.dropout(M, N, y, N, dx, N, 0.2, 8, 1, step=step)
        step.add_(10)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want, keep = _want(torch, x, None, "bf16", 0.2, 8, 1 + 10 * i)
        assert torch.equal(y, want)
        assert torch.equal(dx, _want(torch, want, None, "bf16", 0.2, 8, 1 + 10 * i)[0])
        other = torch.empty_like(x)
        igc.dropout(M, N, x, N, other, N, 0.2, 8, 1, step=step)
        torch.cuda.synchronize()
    assert int(step) == 40


def test_rows_far_down(torch, igc):  # noqa: F811
    """Row numbers and chunk counts past 2^31 elements: the last rows of a matrix of 2^32 + elements."""
    M, N = 2 ** 29 + 3, 9
    x = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    igc.dropout(M, N, x, N, x, N, 0.5, 21)
    for first in (0, 2 ** 28 - 2, M - 5):
        w = words(5, N, 21, 0, first_row=first)
        assert np.array_equal((x[first:first + 5] != 0).cpu().numpy(), w >= 2 ** 31)
