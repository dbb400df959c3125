"""The entry points of the row operators and of the products in 8 bits without a GPU: bad arguments are rejected
with the documented status codes before any HIP call, and the binding's numbers
arrive whole."""
from __future__ import annotations

import ctypes
import math

import pytest

from test_ffn_abi import P, _rejects, igc  # noqa: F401

MOST = 2 ** 31 - 4096


def test_layer_norm_forward_refuses(igc):  # noqa: F811
    good = dict(M=4, N=6, X=P, ldx=6, Y=P, ldy=6, gamma=P, beta=P, mean=P, rstd=P, Q=P, ldq=6, scale=P, type=igc.IGC_F16)
    _rejects(igc, igc.layer_norm_forward, good, [
        dict(M=-1), dict(N=-1), dict(type=igc.IGC_F32), dict(type=7), dict(x_type=igc.IGC_BF16), dict(x_type=3), dict(eps=-1e-5),
        dict(eps=math.nan), dict(eps=math.inf), dict(X=None), dict(ldx=5), dict(ldy=5), dict(ldq=5), dict(X=P + 1), dict(Y=P + 1),
        dict(x_type=igc.IGC_F32, X=P + 2), dict(gamma=P + 2), dict(beta=P + 1), dict(mean=P + 2), dict(rstd=P + 2), dict(scale=None),
        dict(scale=P + 2), dict(Y=None, Q=None, mean=None, rstd=None)])
    assert igc.layer_norm_forward(**{**good, "M": 0, "X": None, "Y": None}, check=False) == igc.IGC_OK
    with pytest.raises(igc.IGCError, match="leading dimension 5 of X"):
        igc.layer_norm_forward(**{**good, "ldx": 5})


def test_layer_norm_backward_refuses(igc):  # noqa: F811
    good = dict(M=4, N=6, dY=P, lddy=6, X=P, ldx=6, mean=P, rstd=P, gamma=P, R=P, ldr=6, dX=P, lddx=6, dgamma=P, dbeta=P, type=igc.IGC_BF16)
    bad = [dict(M=-1), dict(N=-1), dict(type=igc.IGC_F32), dict(x_type=igc.IGC_F16), dict(dX=None, dgamma=None, dbeta=None), dict(dY=None),
           dict(X=None), dict(mean=None), dict(rstd=None), dict(lddy=5), dict(ldx=5), dict(ldr=5), dict(lddx=5), dict(dY=P + 1),
           dict(X=P + 1), dict(R=P + 1), dict(dX=P + 1), dict(x_type=igc.IGC_F32, dX=P + 2), dict(mean=P + 2), dict(gamma=P + 1),
           dict(dgamma=P + 2), dict(dbeta=P + 2)]
    _rejects(igc, igc.layer_norm_backward, good, bad)
    for change in bad:
        with pytest.raises(igc.IGCError) as e:
            igc.layer_norm_backward_workspace_size(**{**good, **change})
        assert e.value.status == igc.IGC_EINVAL
    assert igc.layer_norm_backward(**{**good, "N": 0}, check=False) == igc.IGC_OK
    assert igc.layer_norm_backward_workspace_size(**{**good, "N": 0}) == 0


def test_dropout_refuses(igc):  # noqa: F811
    good = dict(M=4, N=6, X=P, ldx=6, Y=P, ldy=6, p=0.5, seed=1, R=P, ldr=6, step=P, type=igc.IGC_F16)
    _rejects(igc, igc.dropout, good, [
        dict(M=-1), dict(N=-1), dict(type=3), dict(type=-1), dict(y_type=igc.IGC_BF16), dict(y_type=9), dict(p=-0.1), dict(p=1.5),
        dict(p=math.nan), dict(X=None), dict(Y=None), dict(ldx=5), dict(ldy=5), dict(ldr=5), dict(X=P + 1), dict(Y=P + 1), dict(R=P + 1),
        dict(y_type=igc.IGC_F32, Y=P + 2), dict(y_type=igc.IGC_F32, R=P + 2), dict(type=igc.IGC_F32, X=P + 2), dict(step=P + 4)])
    assert igc.dropout(**{**good, "M": 0, "X": None, "Y": None}, check=False) == igc.IGC_OK
    assert igc.dropout(**{**good, "N": 0, "X": None, "Y": None}, check=False) == igc.IGC_OK


def test_quantize_rows_refuses(igc):  # noqa: F811
    good = dict(M=4, N=6, X=P, ldx=6, Q=P, ldq=6, scale=P, type=igc.IGC_BF16)
    _rejects(igc, igc.quantize_rows, good, [
        dict(M=-1), dict(N=-1), dict(type=igc.IGC_F32), dict(type=4), dict(X=None), dict(Q=None), dict(scale=None), dict(ldx=5), dict(ldq=5),
        dict(X=P + 1), dict(scale=P + 2)])
    assert igc.quantize_rows(**{**good, "M": 0, "X": None, "Q": None, "scale": None}, check=False) == igc.IGC_OK


def test_linear_i8_refuses(igc):  # noqa: F811
    good = dict(M=4, N=6, K=8, X=P, ldx=8, x_scale=P, W=P, ldw=8, w_scale=P, Y=P, ldy=6, bias=P, R=P, ldr=6)
    bad = [dict(M=-1), dict(N=-1), dict(K=-1), dict(act=-1), dict(act=6), dict(y_type=3), dict(y_type=-1), dict(X=None), dict(W=None),
           dict(Y=None), dict(x_scale=None), dict(w_scale=None), dict(ldx=7), dict(ldw=7), dict(ldy=5), dict(ldr=5), dict(Y=P + 1),
           dict(y_type=igc.IGC_F32, Y=P + 2), dict(R=P + 1), dict(x_scale=P + 2), dict(w_scale=P + 1), dict(bias=P + 2)]
    _rejects(igc, igc.linear_i8, good, bad)
    for change in bad:
        with pytest.raises(igc.IGCError) as e:
            igc.linear_i8_workspace_size(**{**good, **change})
        assert e.value.status == igc.IGC_EINVAL
    long = {**good, "K": 131072, "ldx": 131072, "ldw": 131072}
    assert igc.linear_i8(**long, check=False) == igc.IGC_EOVERFLOW and "131071" in igc.last_error()
    assert igc.linear_i8(**{**good, "M": 0, "X": None, "x_scale": None, "Y": None}, check=False) == igc.IGC_OK
    assert igc.linear_i8(**{**good, "N": 0, "W": None, "w_scale": None, "Y": None}, check=False) == igc.IGC_OK
    assert igc.linear_i8_workspace_size(**{**good, "M": 0}) == 0


def test_glu_i8_refuses(igc):  # noqa: F811
    good = dict(M=4, N=6, K=8, X=P, ldx=8, x_scale=P, Wg=P, ldwg=8, wg_scale=P, Wu=P, ldwu=8, wu_scale=P, H=P, ldh=6, bias_g=P, bias_u=P)
    bad = [dict(M=-1), dict(N=-1), dict(K=-1), dict(act=6), dict(type=igc.IGC_F32), dict(type=5), dict(X=None), dict(Wg=None), dict(Wu=None),
           dict(H=None), dict(x_scale=None), dict(wg_scale=None), dict(wu_scale=None), dict(ldx=7), dict(ldwg=7), dict(ldwu=7), dict(ldh=5),
           dict(H=P + 1), dict(x_scale=P + 2), dict(wg_scale=P + 2), dict(wu_scale=P + 1), dict(bias_g=P + 1), dict(bias_u=P + 2)]
    _rejects(igc, igc.glu_i8, good, bad)
    long = {**good, "K": 131072, "ldx": 131072, "ldwg": 131072, "ldwu": 131072}
    assert igc.glu_i8(**long, check=False) == igc.IGC_EOVERFLOW
    assert igc.glu_i8(**{**good, "M": 0, "X": None, "x_scale": None, "H": None}, check=False) == igc.IGC_OK
    assert igc.glu_i8_workspace_size(**{**good, "N": 0}) == 0


def test_null_descriptors_and_query_pointers(igc):  # noqa: F811
    L = igc.load()
    for name in ("layer_norm_forward", "layer_norm_backward", "dropout", "quantize_rows", "linear_i8", "glu_i8"):
        assert getattr(L, name)(None, None) == igc.IGC_EINVAL
    size = ctypes.c_size_t(0)
    for name, d in (("layer_norm_backward", igc.binding.LayerNormBackward()), ("linear_i8", igc.binding.LinearI8()), ("glu_i8", igc.binding.GluI8())):
        assert getattr(L, name + "_workspace_size")(None, ctypes.byref(size)) == igc.IGC_EINVAL
        assert getattr(L, name + "_workspace_size")(ctypes.byref(d), None) == igc.IGC_EINVAL


def test_sizes_past_the_index_arithmetic(igc):  # noqa: F811
    ld = 2 ** 31 - 1
    calls = {
        "layer_norm_forward": dict(M=4, N=6, X=P, ldx=ld, Y=P, ldy=ld),
        "layer_norm_backward": dict(M=4, N=6, dY=P, lddy=ld, X=P, ldx=ld, mean=P, rstd=P, dX=P, lddx=ld),
        "dropout": dict(M=4, N=6, X=P, ldx=ld, Y=P, ldy=ld, p=0.5, seed=0),
        "quantize_rows": dict(M=4, N=6, X=P, ldx=ld, Q=P, ldq=ld, scale=P),
        "linear_i8": dict(M=4, N=6, K=8, X=P, ldx=ld, x_scale=P, W=P, ldw=ld, w_scale=P, Y=P, ldy=ld),
        "glu_i8": dict(M=4, N=6, K=8, X=P, ldx=ld, x_scale=P, Wg=P, ldwg=ld, wg_scale=P, Wu=P, ldwu=ld, wu_scale=P, H=P, ldh=ld),
    }
    for name, good in calls.items():
        for axis in "MN":
            for n in (MOST + 1, 2 ** 31 - 1):
                assert getattr(igc, name)(**{**good, axis: n}, check=False) == igc.IGC_EUNSUPPORTED, (name, axis, n)


@pytest.mark.parametrize("native", [True, False], ids=["marshal", "ctypes"])
def test_numbers_of_the_descriptors(igc, monkeypatch, native):  # noqa: F811
    """Every field arrives: checked where a refusal names it, and numbers that do not fit are refused."""
    if not native:
        monkeypatch.setattr(igc.binding, "_native", False)
    drop = dict(M=0, N=6, X=P, ldx=6, Y=P, ldy=6, p=0.5, seed=2 ** 64 - 1, offset=2 ** 64 - 1, stream=0)
    assert igc.dropout(**drop) == igc.IGC_OK
    for change in (dict(seed=-1), dict(seed=2 ** 64), dict(offset=2 ** 64), dict(M=2 ** 32)):
        with pytest.raises(OverflowError):
            igc.dropout(**{**drop, **change})
    for change in (dict(seed=0.5), dict(p="x"), dict(X="x")):
        with pytest.raises((TypeError, ValueError)):
            igc.dropout(**{**drop, **change})
    assert igc.dropout(**{**drop, "p": 2.0}, check=False) == igc.IGC_EINVAL and "p must" in igc.last_error()
    assert igc.dropout(**{**drop, "M": 1, "step": P + 4}, check=False) == igc.IGC_EINVAL and "step" in igc.last_error()
    assert igc.dropout(**{**drop, "M": 1, "ldy": 5}, check=False) == igc.IGC_EINVAL and "5 of Y" in igc.last_error()
    norm = dict(M=0, N=6, X=P, ldx=6, Y=P, ldy=6, stream=0)
    assert igc.layer_norm_forward(**norm) == igc.IGC_OK
    assert igc.layer_norm_forward(**norm, eps=-1.0, check=False) == igc.IGC_EINVAL and "eps" in igc.last_error()
    assert igc.layer_norm_forward(**norm, Q=P, ldq=6, check=False) == igc.IGC_EINVAL and "scale" in igc.last_error()
    assert igc.quantize_rows(1, 6, P, 6, P, 5, P, stream=0, check=False) == igc.IGC_EINVAL and "5 of Q" in igc.last_error()


def test_structures_match_the_header(igc):  # noqa: F811
    """The descriptors' fields, in the header's order and types."""
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "igc.h")).read()
    kinds = {"int": ctypes.c_int, "float": ctypes.c_float, "double": ctypes.c_double, "uint64_t": ctypes.c_uint64, "size_t": ctypes.c_size_t}
    for name, desc in igc.binding._DESCRIPTORS.items():
        body = re.search(r"typedef struct igc_%s \{(.*?)\} igc_%s;" % (name, name), text, re.S).group(1)
        fields = []
        for line in filter(None, (l.strip() for l in body.split(";"))):
            kind, names = re.fullmatch(r"((?:const )?\w+(?: long)?(?:\s*\*(?: const\s*\*)?)?)\s*(.*)", line, re.S).groups()
            for n in names.split(","):
                star = "*" in kind or "*" in n
                fields.append((n.strip().lstrip("* "), ctypes.c_void_p if star else kinds[kind.strip()]))
        assert fields == list(desc._fields_), name
