"""Thin ctypes binding of libigc.so (include/igc.h).

Argument marshalling only: every computation runs in the library's HIP
kernels.  Device buffers are passed either as raw device addresses (ints) or
as torch tensors on a ROCm device (their ``data_ptr()`` is taken); streams as
a raw ``hipStream_t`` (int) or a ``torch.cuda.Stream``.  When no stream is
given, torch's current stream is used if torch is loaded, else the null
stream.

The feed-forward entry points fill their descriptors in a small extension
module (``_marshal``, csrc/marshal.cpp) where torch is installed.

The library must already be built (``python -m implicit_gemm_convolution_amd.build``
or ``__graft_entry__.build()``); a missing library raises, there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import operator
import os
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libigc.so")

IGC_OK = 0
IGC_EINVAL = -1
IGC_EUNSUPPORTED = -2
IGC_EOVERFLOW = -3
IGC_EHIP = -4
IGC_ENODEV = -5

# Element types and activations of the feed-forward operators.
IGC_F16 = 0
IGC_BF16 = 1
IGC_F32 = 2
IGC_ACT_NONE = 0
IGC_ACT_RELU = 1
IGC_ACT_GELU = 2
IGC_ACT_GELU_TANH = 3
IGC_ACT_SILU = 4
IGC_ACT_SIGMOID = 5

# Every symbol include/igc.h declares.
EXPORTED = ("gemm_f16f32", "gemm_u8i8_zp", "conv2d_implicit_gemm", "conv2d_u8i8_zp",
            "gemm_f16f32_workspace_size", "gemm_u8i8_zp_workspace_size",
            "conv2d_implicit_gemm_workspace_size", "conv2d_u8i8_zp_workspace_size",
            "gemm_f16f32_noalloc", "conv2d_implicit_gemm_nhwcnc", "conv2d_implicit_gemm_nhwcnc_workspace_size",
            "u8i8_colsum",
            "linear_forward", "linear_forward_workspace_size", "linear_backward", "linear_backward_workspace_size",
            "glu_forward", "glu_forward_workspace_size", "glu_backward", "glu_backward_workspace_size",
            "grad_clip", "grad_clip_workspace_size",
            "igc_status_string", "igc_last_error", "igc_device_check", "igc_set_tuning")


class IGCError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({detail})")


class Epilogue(ctypes.Structure):
    """igc_u8i8_epilogue."""
    _fields_ = [
        ("C_i32", ctypes.c_void_p),
        ("ldc", ctypes.c_int),
        ("D_f32", ctypes.c_void_p),
        ("ldd", ctypes.c_int),
        ("dq_scale", ctypes.c_float),
        ("Q_i8", ctypes.c_void_p),
        ("ldq", ctypes.c_int),
        ("scale_n", ctypes.c_void_p),
        ("bias_n", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_size_t),
        ("colsum_B", ctypes.c_void_p),
    ]


def _fields(text):
    """Structure fields from "name:kind" words: i int, p pointer, f float, z size_t."""
    kinds = {"i": ctypes.c_int, "p": ctypes.c_void_p, "f": ctypes.c_float, "z": ctypes.c_size_t}
    return [(w.split(":")[0], kinds[w.split(":")[1]]) for w in text.split()]


class LinearForward(ctypes.Structure):
    """igc_linear_forward."""
    _fields_ = _fields("M:i N:i K:i type:i act:i y_type:i X:p ldx:i W:p ldw:i bias:p R:p ldr:i Y:p ldy:i Z:p ldz:i "
                       "workspace:p ws_bytes:z")


class LinearBackward(ctypes.Structure):
    """igc_linear_backward."""
    _fields_ = _fields("M:i N:i K:i type:i act:i dY:p lddy:i Z:p ldz:i X:p ldx:i W:p ldw:i dX:p lddx:i dW:p lddw:i "
                       "dbias:p workspace:p ws_bytes:z")


class GluForward(ctypes.Structure):
    """igc_glu_forward."""
    _fields_ = _fields("M:i N:i K:i type:i act:i X:p ldx:i Wg:p ldwg:i Wu:p ldwu:i bias_g:p bias_u:p H:p ldh:i "
                       "G:p ldg:i U:p ldu:i workspace:p ws_bytes:z")


class GluBackward(ctypes.Structure):
    """igc_glu_backward."""
    _fields_ = _fields("M:i N:i K:i type:i act:i dH:p lddh:i G:p ldg:i U:p ldu:i X:p ldx:i Wg:p ldwg:i Wu:p ldwu:i "
                       "dX:p lddx:i dWg:p lddwg:i dWu:p lddwu:i dbias_g:p dbias_u:p workspace:p ws_bytes:z")


class GradClip(ctypes.Structure):
    """igc_grad_clip."""
    _fields_ = _fields("count:i grads:p outs:p sizes:p types:p max_norm:f norm:p workspace:p ws_bytes:z")


# The entry points that take a descriptor: its structure, and for _marshal
# its fields before the workspace.
_DESCRIPTORS = {"linear_forward": LinearForward, "linear_backward": LinearBackward, "glu_forward": GluForward,
                "glu_backward": GluBackward, "grad_clip": GradClip}
_FORMATS = {name: "".join("i" if kind is ctypes.c_int else "p" for _, kind in desc._fields_[:-2])
            for name, desc in _DESCRIPTORS.items()}

_lib = None


def load() -> ctypes.CDLL:
    """Load libigc.so once.  torch (when installed) is imported first so that
    the library binds to the HIP runtime torch already uses."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FileNotFoundError(
            f"{LIB_PATH} is not built; run `python -m implicit_gemm_convolution_amd.build`")
    try:  # one HIP runtime per process: let torch's copy be the one that is loaded
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    i, p, z = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    pz = ctypes.POINTER(ctypes.c_size_t)
    L.gemm_f16f32.argtypes = [i, i, i, p, i, p, i, p, i, p, z, p]
    L.gemm_f16f32.restype = i
    L.gemm_f16f32_noalloc.argtypes = [i, i, i, p, i, p, i, p, i, p]
    L.gemm_f16f32_noalloc.restype = i
    L.gemm_u8i8_zp.argtypes = [i, i, i, p, i, i, p, i, i, ctypes.POINTER(Epilogue), p]
    L.gemm_u8i8_zp.restype = i
    L.conv2d_implicit_gemm.argtypes = [i] * 11 + [p, p, p, p, z, p]
    L.conv2d_implicit_gemm.restype = i
    L.conv2d_u8i8_zp.argtypes = [i] * 11 + [p, i, p, i, ctypes.POINTER(Epilogue), p]
    L.conv2d_implicit_gemm_nhwcnc.argtypes = [i] * 11 + [p, p, p, p, z, p]
    L.conv2d_implicit_gemm_nhwcnc.restype = i
    L.conv2d_u8i8_zp.restype = i
    for name in ("gemm_f16f32_workspace_size", "gemm_u8i8_zp_workspace_size"):
        getattr(L, name).argtypes = [i, i, i, pz]
        getattr(L, name).restype = i
    for name in ("conv2d_implicit_gemm_workspace_size", "conv2d_u8i8_zp_workspace_size",
                 "conv2d_implicit_gemm_nhwcnc_workspace_size"):
        getattr(L, name).argtypes = [i] * 11 + [pz]
        getattr(L, name).restype = i
    L.u8i8_colsum.argtypes = [i, i, p, i, p, p]
    L.u8i8_colsum.restype = i
    for name, desc in _DESCRIPTORS.items():
        getattr(L, name).argtypes = [ctypes.POINTER(desc), p]
        getattr(L, name).restype = i
        getattr(L, name + "_workspace_size").argtypes = [ctypes.POINTER(desc), pz]
        getattr(L, name + "_workspace_size").restype = i
    L.igc_set_tuning.argtypes = [i, i]
    L.igc_set_tuning.restype = i
    L.igc_status_string.argtypes = [i]
    L.igc_status_string.restype = ctypes.c_char_p
    L.igc_last_error.argtypes = []
    L.igc_last_error.restype = ctypes.c_char_p
    L.igc_device_check.argtypes = []
    L.igc_device_check.restype = i
    _lib = L
    return L


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    raise TypeError(f"expected a device address or a tensor, got {type(x)}")


_raw_stream = None  # torch's current stream as a raw hipStream_t, found at the first call


def _current_stream() -> int:
    """torch's current stream.  Looked up by every call, so through the raw
    getter where torch has it (0.2 us; a Stream object costs 3)."""
    global _raw_stream
    torch = sys.modules["torch"]
    if _raw_stream is None:
        get, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if get is not None and device is not None:
            torch.cuda.init()
            _raw_stream = lambda: get(device())  # noqa: E731
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return int(_raw_stream())


def _stream(s) -> int | None:
    if s is None:
        if _raw_stream is not None:
            return _current_stream()
        torch = sys.modules.get("torch")
        if torch is not None and torch.cuda.is_available():
            return _current_stream()
        return None
    if isinstance(s, int):
        return s
    if hasattr(s, "cuda_stream"):
        return int(s.cuda_stream)
    raise TypeError(f"expected a hipStream_t or a torch stream, got {type(s)}")


def _check(status: int, where: str) -> int:
    if status != IGC_OK:
        L = load()
        detail = L.igc_last_error().decode() or L.igc_status_string(status).decode()
        raise IGCError(status, where, detail)
    return status


def status_string(status: int) -> str:
    return load().igc_status_string(status).decode()


def last_error() -> str:
    return load().igc_last_error().decode()


def device_check(raise_on_error: bool = False) -> int:
    st = load().igc_device_check()
    return _check(st, "igc_device_check") if raise_on_error else st


def set_tuning(force_variant: int = -1, streamk_mode: int = 1, *, check=True) -> int:
    """Process-wide overrides (tests, sweeps): a forced tile variant (-1 = by
    shape) and the stream-K mode (0 off, 1 where it pays, 2 always)."""
    st = load().igc_set_tuning(int(force_variant), int(streamk_mode))
    return _check(st, "igc_set_tuning") if check else st


def _ws_query(name, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(getattr(load(), name)(*args, ctypes.byref(out)), name)
    return int(out.value)


def gemm_f16f32_workspace_size(M, N, K) -> int:
    return _ws_query("gemm_f16f32_workspace_size", M, N, K)


def gemm_u8i8_zp_workspace_size(M, N, K) -> int:
    return _ws_query("gemm_u8i8_zp_workspace_size", M, N, K)


def conv2d_implicit_gemm_workspace_size(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w) -> int:
    return _ws_query("conv2d_implicit_gemm_workspace_size", Nb, H, W, C, Kout, R, S, stride_h, stride_w,
                     pad_h, pad_w)


def conv2d_u8i8_zp_workspace_size(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w) -> int:
    return _ws_query("conv2d_u8i8_zp_workspace_size", Nb, H, W, C, Kout, R, S, stride_h, stride_w,
                     pad_h, pad_w)


def conv2d_implicit_gemm_nhwcnc_workspace_size(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w) -> int:
    return _ws_query("conv2d_implicit_gemm_nhwcnc_workspace_size", Nb, H, W, C, Kout, R, S, stride_h, stride_w,
                     pad_h, pad_w)


def _ws_bytes(workspace, ws_bytes):
    if ws_bytes is None:
        ws_bytes = int(workspace.numel() * workspace.element_size()) if hasattr(workspace, "numel") else 0
    return ws_bytes


def gemm_f16f32(M, N, K, A, lda, B, ldb, C, ldc, stream=None, *, workspace=None, ws_bytes=None,
                check=True) -> int:
    st = load().gemm_f16f32(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, _addr(workspace),
                            _ws_bytes(workspace, ws_bytes), _stream(stream))
    return _check(st, "gemm_f16f32") if check else st


def gemm_f16f32_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=None, *, check=True) -> int:
    """gemm_f16f32 with its workspace in the library's static device array
    (allocates nothing; calls that overlap on one GPU race)."""
    st = load().gemm_f16f32_noalloc(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, _stream(stream))
    return _check(st, "gemm_f16f32_noalloc") if check else st


def u8i8_colsum(N, K, B, ldb, colsum, stream=None, *, check=True) -> int:
    """colsum[n] = sum_k B[n*ldb + k] (int32), for the colsum_B argument."""
    st = load().u8i8_colsum(N, K, _addr(B), ldb, _addr(colsum), _stream(stream))
    return _check(st, "u8i8_colsum") if check else st


def gemm_u8i8_zp(M, N, K, A, lda, zA, B, ldb, zB, *, C_i32=None, ldc=0, D_f32=None, ldd=0,
                 dq_scale=0.0, Q_i8=None, ldq=0, scale_n=None, bias_n=None, stream=None,
                 workspace=None, ws_bytes=None, colsum_B=None, check=True) -> int:
    ep = Epilogue(_addr(C_i32), ldc, _addr(D_f32), ldd, float(dq_scale), _addr(Q_i8), ldq,
                  _addr(scale_n), _addr(bias_n), _addr(workspace), _ws_bytes(workspace, ws_bytes),
                  _addr(colsum_B))
    st = load().gemm_u8i8_zp(M, N, K, _addr(A), lda, zA, _addr(B), ldb, zB, ctypes.byref(ep),
                             _stream(stream))
    return _check(st, "gemm_u8i8_zp") if check else st


def conv2d_implicit_gemm(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w, x, w, y,
                         stream=None, *, workspace=None, ws_bytes=None, check=True) -> int:
    st = load().conv2d_implicit_gemm(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w,
                                     _addr(x), _addr(w), _addr(y), _addr(workspace),
                                     _ws_bytes(workspace, ws_bytes), _stream(stream))
    return _check(st, "conv2d_implicit_gemm") if check else st


def conv2d_implicit_gemm_nhwcnc(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w, x, w, y,
                                stream=None, *, workspace=None, ws_bytes=None, check=True) -> int:
    """The convolution on blocked NHWCnc tensors (block 16); the workspace is required."""
    st = load().conv2d_implicit_gemm_nhwcnc(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w,
                                            _addr(x), _addr(w), _addr(y), _addr(workspace),
                                            _ws_bytes(workspace, ws_bytes), _stream(stream))
    return _check(st, "conv2d_implicit_gemm_nhwcnc") if check else st


def conv2d_u8i8_zp(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w, x, zA, w, zB, *,
                   C_i32=None, ldc=0, D_f32=None, ldd=0, dq_scale=0.0, Q_i8=None, ldq=0,
                   scale_n=None, bias_n=None, stream=None, workspace=None, ws_bytes=None,
                   colsum_B=None, check=True) -> int:
    ep = Epilogue(_addr(C_i32), ldc, _addr(D_f32), ldd, float(dq_scale), _addr(Q_i8), ldq,
                  _addr(scale_n), _addr(bias_n), _addr(workspace), _ws_bytes(workspace, ws_bytes),
                  _addr(colsum_B))
    st = load().conv2d_u8i8_zp(Nb, H, W, C, Kout, R, S, stride_h, stride_w, pad_h, pad_w, _addr(x), zA,
                               _addr(w), zB, ctypes.byref(ep), _stream(stream))
    return _check(st, "conv2d_u8i8_zp") if check else st


# ---------------------------------------------------------------------------
# The feed-forward operators.  Each <entry>_workspace_size takes the entry's
# arguments (but for workspace and stream) and returns the bytes that the
# call needs.
# ---------------------------------------------------------------------------
_native = None   # the _marshal module; False without torch
_entries = None  # (the library, addresses of its entry points)


def _marshal():
    global _native
    if _native is None:
        load()
        try:
            import torch  # noqa: F401
        except ImportError:
            _native = False
        else:
            from . import _marshal as native
            _native = native
    return _native


def _entry(name) -> int:
    """An entry point's address."""
    global _entries
    L = load()
    if _entries is None or _entries[0] is not L:
        _entries = L, {n + q: ctypes.cast(getattr(L, n + q), ctypes.c_void_p).value
                       for n in _DESCRIPTORS for q in ("", "_workspace_size")}
    return _entries[1][name]


def _int32(v) -> int:
    """A whole number that an int of the descriptor holds (ctypes would cut it to 32 bits)."""
    v = operator.index(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise OverflowError("%d does not fit in 32 bits" % v)
    return v


def _describe(name, fields, workspace, ws_bytes):
    """The entry point's descriptor."""
    values = [_addr(v) if kind == "p" else _int32(v) for kind, v in zip(_FORMATS[name], fields)]
    return _DESCRIPTORS[name](*values, _addr(workspace), _ws_bytes(workspace, ws_bytes))


def _call(name, check, stream, workspace, ws_bytes, *fields) -> int:
    native = _native if _native is not None else _marshal()
    if native:
        st = native.call(_entry(name), _FORMATS[name], _stream(stream), workspace, ws_bytes, *fields)
    else:
        st = getattr(load(), name)(_describe(name, fields, workspace, ws_bytes), _stream(stream))
    return _check(st, name) if check else st


def _query(name, *fields) -> int:
    return _ws_query(name + "_workspace_size", _describe(name, fields, None, 0))


def linear_forward(M, N, K, X, ldx, W, ldw, Y, ldy, *, type=IGC_BF16, act=IGC_ACT_NONE, y_type=None, bias=None, R=None, ldr=0,
                   Z=None, ldz=0, stream=None, workspace=None, ws_bytes=None, check=True) -> int:
    """Z = X W^T + bias; Y = act(Z) + R (y_type None: the operands' type)."""
    return _call("linear_forward", check, stream, workspace, ws_bytes,
                 M, N, K, type, act, type if y_type is None else y_type, X, ldx, W, ldw, bias, R, ldr, Y, ldy, Z, ldz)


def linear_forward_workspace_size(M, N, K, X, ldx, W, ldw, Y, ldy, *, type=IGC_BF16, act=IGC_ACT_NONE, y_type=None, bias=None,
                                  R=None, ldr=0, Z=None, ldz=0) -> int:
    return _query("linear_forward", M, N, K, type, act, type if y_type is None else y_type, X, ldx, W, ldw, bias, R, ldr,
                  Y, ldy, Z, ldz)


def linear_backward(M, N, K, dY, lddy, *, Z=None, ldz=0, X=None, ldx=0, W=None, ldw=0, dX=None, lddx=0, dW=None, lddw=0,
                    dbias=None, type=IGC_BF16, act=IGC_ACT_NONE, stream=None, workspace=None, ws_bytes=None, check=True) -> int:
    """D = dY act'(Z); dX = D W; dW = D^T X; dbias = column sums of D (any subset)."""
    return _call("linear_backward", check, stream, workspace, ws_bytes,
                 M, N, K, type, act, dY, lddy, Z, ldz, X, ldx, W, ldw, dX, lddx, dW, lddw, dbias)


def linear_backward_workspace_size(M, N, K, dY, lddy, *, Z=None, ldz=0, X=None, ldx=0, W=None, ldw=0, dX=None, lddx=0, dW=None,
                                   lddw=0, dbias=None, type=IGC_BF16, act=IGC_ACT_NONE) -> int:
    return _query("linear_backward", M, N, K, type, act, dY, lddy, Z, ldz, X, ldx, W, ldw, dX, lddx, dW, lddw, dbias)


def glu_forward(M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, H, ldh, *, bias_g=None, bias_u=None, G=None, ldg=0, U=None, ldu=0,
                type=IGC_BF16, act=IGC_ACT_SILU, stream=None, workspace=None, ws_bytes=None, check=True) -> int:
    """G = X Wg^T + bias_g; U = X Wu^T + bias_u; H = act(G) U."""
    return _call("glu_forward", check, stream, workspace, ws_bytes,
                 M, N, K, type, act, X, ldx, Wg, ldwg, Wu, ldwu, bias_g, bias_u, H, ldh, G, ldg, U, ldu)


def glu_forward_workspace_size(M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, H, ldh, *, bias_g=None, bias_u=None, G=None, ldg=0, U=None,
                               ldu=0, type=IGC_BF16, act=IGC_ACT_SILU) -> int:
    return _query("glu_forward", M, N, K, type, act, X, ldx, Wg, ldwg, Wu, ldwu, bias_g, bias_u, H, ldh, G, ldg, U, ldu)


def glu_backward(M, N, K, dH, lddh, G, ldg, U, ldu, *, X=None, ldx=0, Wg=None, ldwg=0, Wu=None, ldwu=0, dX=None, lddx=0,
                 dWg=None, lddwg=0, dWu=None, lddwu=0, dbias_g=None, dbias_u=None, type=IGC_BF16, act=IGC_ACT_SILU,
                 stream=None, workspace=None, ws_bytes=None, check=True) -> int:
    """dU = dH act(G), dG = dH U act'(G); dX = dG Wg + dU Wu; dW* = d*^T X; dbias_* = column sums (any subset)."""
    return _call("glu_backward", check, stream, workspace, ws_bytes,
                 M, N, K, type, act, dH, lddh, G, ldg, U, ldu, X, ldx, Wg, ldwg, Wu, ldwu, dX, lddx, dWg, lddwg, dWu, lddwu,
                 dbias_g, dbias_u)


def glu_backward_workspace_size(M, N, K, dH, lddh, G, ldg, U, ldu, *, X=None, ldx=0, Wg=None, ldwg=0, Wu=None, ldwu=0, dX=None,
                                lddx=0, dWg=None, lddwg=0, dWu=None, lddwu=0, dbias_g=None, dbias_u=None, type=IGC_BF16,
                                act=IGC_ACT_SILU) -> int:
    return _query("glu_backward", M, N, K, type, act, dH, lddh, G, ldg, U, ldu, X, ldx, Wg, ldwg, Wu, ldwu, dX, lddx, dWg, lddwg,
                  dWu, lddwu, dbias_g, dbias_u)


def _clip(entry, query, stream, workspace, ws_bytes, grads, out, max_norm, norm):
    native = _marshal()
    if not native:
        raise RuntimeError("grad_clip takes torch tensors, and torch is not installed")
    return native.clip(_entry(entry), query, stream, workspace, ws_bytes, grads, out, max_norm, norm)


def grad_clip(grads, max_norm, norm, *, out=None, stream=None, workspace=None, ws_bytes=None, check=True) -> int:
    """norm = the global norm of `grads` (contiguous fp16 / bf16 / fp32 tensors); out = grads * min(1, max_norm / (norm + 1e-6)),
    in place without `out`."""
    st = _clip("grad_clip", False, _stream(stream), workspace, ws_bytes, grads, out, max_norm, norm)
    return _check(st, "grad_clip") if check else st


def grad_clip_workspace_size(grads, max_norm, norm, *, out=None) -> int:
    st, size = _clip("grad_clip_workspace_size", True, None, None, None, grads, out, max_norm, norm)
    _check(st, "grad_clip_workspace_size")
    return size
