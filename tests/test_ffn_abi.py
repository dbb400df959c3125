"""The feed-forward entry points without a GPU: bad arguments are rejected with
the documented status codes before any HIP call, and the binding checks its
tensors."""
from __future__ import annotations

import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def igc():
    import implicit_gemm_convolution_amd as m

    if not os.path.exists(m.LIB_PATH):
        from implicit_gemm_convolution_amd import build

        build.build()
    m.load()
    return m


def _rejects(igc, f, good, bad):
    """Each change of `bad` turns the call `good` into one that is refused."""
    for change in bad:
        st = f(**{**good, **change}, check=False)
        assert st == igc.IGC_EINVAL, change
        assert igc.last_error()


P = 4096  # an address that is never read: every call here is refused or empty


def test_linear_forward_refuses(igc):
    good = dict(M=4, N=6, K=8, X=P, ldx=8, W=P, ldw=8, Y=P, ldy=6, type=igc.IGC_F16, act=igc.IGC_ACT_GELU)
    _rejects(igc, igc.linear_forward, good, [
        dict(M=-1), dict(N=-1), dict(K=-1), dict(type=igc.IGC_F32), dict(type=7), dict(act=-1), dict(act=6),
        dict(y_type=igc.IGC_BF16), dict(X=None), dict(W=None), dict(Y=None), dict(ldx=7), dict(ldw=7), dict(ldy=5),
        dict(X=P + 1), dict(W=P + 1), dict(Y=P + 1), dict(y_type=igc.IGC_F32, Y=P + 2), dict(R=P, ldr=5), dict(R=P + 1, ldr=6),
        dict(Z=P, ldz=5), dict(Z=P + 1, ldz=6), dict(bias=P + 2)])
    assert igc.linear_forward(**{**good, "M": 0, "X": None, "Y": None}, check=False) == igc.IGC_OK
    assert igc.linear_forward(**{**good, "N": 0, "W": None, "Y": None}, check=False) == igc.IGC_OK
    with pytest.raises(igc.IGCError, match="ldx|leading dimension 7 of X"):
        igc.linear_forward(**{**good, "ldx": 7})


def test_linear_backward_refuses(igc):
    good = dict(M=4, N=6, K=8, dY=P, lddy=6, Z=P, ldz=6, X=P, ldx=8, W=P, ldw=8, dX=P, lddx=8, dW=P, lddw=8, dbias=P,
                type=igc.IGC_BF16, act=igc.IGC_ACT_SILU)
    _rejects(igc, igc.linear_backward, good, [
        dict(M=-1), dict(type=igc.IGC_F32), dict(act=9), dict(dX=None, dW=None, dbias=None), dict(dY=None), dict(Z=None),
        dict(X=None), dict(W=None), dict(lddy=5), dict(ldz=5), dict(ldx=7), dict(ldw=7), dict(lddx=7), dict(lddw=7),
        dict(dY=P + 1), dict(Z=P + 1), dict(dX=P + 1), dict(dW=P + 1), dict(dbias=P + 2)])


def test_glu_forward_refuses(igc):
    good = dict(M=4, N=6, K=8, X=P, ldx=8, Wg=P, ldwg=8, Wu=P, ldwu=8, H=P, ldh=6, type=igc.IGC_BF16)
    _rejects(igc, igc.glu_forward, good, [
        dict(K=-2), dict(type=igc.IGC_F32), dict(act=6), dict(X=None), dict(Wg=None), dict(Wu=None), dict(H=None),
        dict(ldx=7), dict(ldwg=7), dict(ldwu=7), dict(ldh=5), dict(G=P, ldg=5), dict(U=P, ldu=5), dict(Wu=P + 1),
        dict(bias_g=P + 1), dict(bias_u=P + 2)])
    assert igc.glu_forward(**{**good, "M": 0, "X": None, "H": None}, check=False) == igc.IGC_OK


def test_glu_backward_refuses(igc):
    good = dict(M=4, N=6, K=8, dH=P, lddh=6, G=P, ldg=6, U=P, ldu=6, X=P, ldx=8, Wg=P, ldwg=8, Wu=P, ldwu=8, dX=P, lddx=8,
                dWg=P, lddwg=8, dWu=P, lddwu=8, dbias_g=P, dbias_u=P, type=igc.IGC_F16)
    _rejects(igc, igc.glu_backward, good, [
        dict(N=-1), dict(type=igc.IGC_F32), dict(act=-1), dict(dX=None, dWg=None, dWu=None, dbias_g=None, dbias_u=None),
        dict(dH=None), dict(G=None), dict(U=None), dict(X=None), dict(Wg=None), dict(Wu=None), dict(lddh=5), dict(ldg=5),
        dict(ldu=5), dict(ldx=7), dict(ldwg=7), dict(ldwu=7), dict(lddx=7), dict(lddwg=7), dict(lddwu=7), dict(dbias_u=P + 1)])


def test_descriptor_and_query_pointers(igc):
    L = igc.load()
    size = ctypes.c_size_t(0)
    for name in ("linear_forward", "linear_backward", "glu_forward", "glu_backward", "grad_clip"):
        assert getattr(L, name)(None, None) == igc.IGC_EINVAL
        assert getattr(L, name + "_workspace_size")(None, ctypes.byref(size)) == igc.IGC_EINVAL
    d = igc.binding.LinearForward()
    assert L.linear_forward_workspace_size(ctypes.byref(d), None) == igc.IGC_EINVAL
    assert L.linear_forward_workspace_size(ctypes.byref(d), ctypes.byref(size)) == igc.IGC_OK and size.value == 0


def _clip(igc, sizes=(4, 4), types=None, ptrs=(P, P), outs=None, count=None, max_norm=1.0, norm=P, arrays=True, ws=P, ws_bytes=1 << 20):
    n = len(sizes)
    types = (igc.IGC_F32,) * n if types is None else types
    a = ctypes.addressof
    g = (ctypes.c_void_p * n)(*ptrs)
    o = None if outs is None else (ctypes.c_void_p * n)(*outs)
    s, t = (ctypes.c_longlong * n)(*sizes), (ctypes.c_int * n)(*types)
    d = igc.binding.GradClip(n if count is None else count, a(g) if arrays else None, a(o) if o else None, a(s), a(t), max_norm,
                             norm, ws, ws_bytes)
    return igc.load().grad_clip(ctypes.byref(d), None)


def test_grad_clip_refuses(igc):
    E = igc.IGC_EINVAL
    assert _clip(igc, count=-1) == E
    assert _clip(igc, max_norm=-1.0) == E
    assert _clip(igc, norm=None) == E
    assert _clip(igc, norm=P + 2) == E
    assert _clip(igc, arrays=False) == E
    assert _clip(igc, sizes=(4, -1)) == E
    assert _clip(igc, types=(igc.IGC_F32, 3)) == E
    assert _clip(igc, ptrs=(P, None)) == E
    assert _clip(igc, ptrs=(P, P + 2)) == E              # an fp32 tensor at a 2-byte address
    assert _clip(igc, outs=(P, P + 1), types=(igc.IGC_F16,) * 2) == E


def test_grad_clip_binding_checks_its_tensors(igc):
    import torch

    norm = torch.zeros(1)
    a, b = torch.zeros(4, 6), torch.zeros(3, dtype=torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        igc.grad_clip([a.t()], 1.0, norm)
    with pytest.raises(ValueError, match="outputs"):
        igc.grad_clip([a, b], 1.0, norm, out=[a])
    with pytest.raises(ValueError, match="type or size"):
        igc.grad_clip([a, b], 1.0, norm, out=[a, torch.zeros(3)])
    with pytest.raises(TypeError, match="float64"):
        igc.grad_clip([a.double()], 1.0, norm)


def test_arguments_of_every_kind(igc):
    """Addresses as ints, tensors, None or anything with data_ptr(); whole numbers that fit; nothing else."""
    import torch

    class Holder:
        def data_ptr(self):
            return P

    good = dict(M=0, N=6, K=8, X=P, ldx=8, W=P, ldw=8, Y=None, ldy=6, stream=0)
    for x in (P, None, torch.zeros(4), Holder()):
        assert igc.linear_forward(**{**good, "X": x}) == igc.IGC_OK
    with pytest.raises(TypeError, match="address or a tensor"):
        igc.linear_forward(**{**good, "X": "text"})
    with pytest.raises(TypeError):
        igc.linear_forward(**{**good, "M": 1.5})
    with pytest.raises(OverflowError):
        igc.linear_forward(**{**good, "ldx": 1 << 40})
    with pytest.raises(RuntimeError):  # a tensor without memory of its own
        igc.linear_forward(**{**good, "X": torch.sparse_coo_tensor(size=(2, 2))})
    with pytest.raises(TypeError, match="tensors"):
        igc.grad_clip([1, 2], 1.0, None, stream=0)


def test_without_torch_the_descriptors_go_through_ctypes(igc, monkeypatch):
    good = dict(M=4, N=6, K=8, X=P, ldx=8, W=P, ldw=8, Y=P, ldy=6, type=igc.IGC_F16, act=igc.IGC_ACT_GELU, stream=0)
    monkeypatch.setattr(igc.binding, "_native", False)
    assert igc.linear_forward(**{**good, "M": 0, "X": None, "Y": None}) == igc.IGC_OK
    _rejects(igc, igc.linear_forward, good, [dict(ldx=7), dict(W=None), dict(Y=P + 1), dict(Z=P, ldz=5), dict(R=P, ldr=5)])
    with pytest.raises(RuntimeError, match="torch"):
        igc.grad_clip([], 1.0, P, stream=0)


def test_sizes_past_the_index_arithmetic(igc):
    """Extents within a tile of 2^31 (2^30 where two matrices lie side by side) are refused, by the calls and the queries."""
    most = 2 ** 31 - 4096
    ld = 2 ** 31 - 1
    lin = dict(M=4, N=6, K=8, dY=P, lddy=ld, Z=P, ldz=ld, X=P, ldx=ld, W=P, ldw=ld, dX=P, lddx=ld, dW=P, lddw=ld, dbias=P, act=igc.IGC_ACT_SILU)
    fwd = dict(M=4, N=6, K=8, X=P, ldx=ld, W=P, ldw=ld, Y=P, ldy=ld)
    glu = dict(M=4, N=6, K=8, X=P, ldx=ld, Wg=P, ldwg=ld, Wu=P, ldwu=ld, H=P, ldh=ld)
    back = dict(M=4, N=6, K=8, dH=P, lddh=ld, G=P, ldg=ld, U=P, ldu=ld, X=P, ldx=ld, Wg=P, ldwg=ld, Wu=P, ldwu=ld, dX=P, lddx=ld,
                dWg=P, lddwg=ld, dWu=P, lddwu=ld)
    for name, good in (("linear_forward", fwd), ("linear_backward", lin), ("glu_forward", glu), ("glu_backward", back)):
        call, query = getattr(igc, name), getattr(igc, name + "_workspace_size")
        for axis in "MNK":
            top = 2 ** 30 - 2048 if (name, axis) == ("glu_backward", "N") else most
            for n in (top + 1, 2 ** 31 - 64, 2 ** 31 - 1):
                bad = {**good, axis: n}
                assert call(**bad, check=False) == igc.IGC_EUNSUPPORTED, (name, axis, n)
                with pytest.raises(igc.IGCError, match=axis) as e:
                    query(**bad)
                assert e.value.status == igc.IGC_EUNSUPPORTED


def test_grad_clip_refuses_tensors_of_another_device_and_norms_of_another_type(igc):
    """Nothing but addresses of the GPU reaches the kernels; the size query reads no tensor and takes any device's."""
    import torch

    a, norm = torch.zeros(4, 6), torch.zeros(1)
    for bad in (torch.zeros(1, dtype=torch.float64), torch.zeros(1, dtype=torch.bfloat16), torch.zeros(0)):
        with pytest.raises(TypeError, match="norm must be a float32"):
            igc.grad_clip([a], 1.0, bad, workspace=P, ws_bytes=1 << 20, stream=0)
    with pytest.raises(TypeError, match="on the GPU, not on cpu"):
        igc.grad_clip([a], 1.0, P, workspace=P, ws_bytes=1 << 20, stream=0)
    with pytest.raises(TypeError, match="on the GPU, not on cpu"):
        igc.grad_clip([], 1.0, norm, workspace=P, ws_bytes=1 << 20, stream=0)
    with pytest.raises(TypeError, match="on the GPU, not on cpu"):
        igc.grad_clip([], 1.0, P, workspace=torch.zeros(1 << 16, dtype=torch.uint8), stream=0)
    assert igc.grad_clip_workspace_size([a], 1.0, norm) > 0


def test_size_queries_take_the_numbers_that_the_calls_take(igc):
    """Whole numbers of any type; one that an int does not hold is not cut to 32 bits."""
    import numpy as np

    good = dict(M=0, N=6, K=8, X=P, ldx=8, W=P, ldw=8, Y=P, ldy=6)
    assert igc.linear_forward_workspace_size(**{**good, "N": np.int64(6), "ldx": np.int32(8)}) == 0
    for bad in (dict(ldx=2 ** 32 + 8), dict(M=2 ** 32), dict(N=-2 ** 31 - 1)):
        with pytest.raises(OverflowError):
            igc.linear_forward_workspace_size(**{**good, **bad})
    with pytest.raises(TypeError):
        igc.linear_forward_workspace_size(**{**good, "M": 0.0})


def test_without_torch_numbers_are_not_cut(igc, monkeypatch):
    monkeypatch.setattr(igc.binding, "_native", False)
    good = dict(M=0, N=6, K=8, X=P, ldx=8, W=P, ldw=8, Y=P, ldy=6, stream=0)
    with pytest.raises(OverflowError):
        igc.linear_forward(**{**good, "M": 2 ** 32})
