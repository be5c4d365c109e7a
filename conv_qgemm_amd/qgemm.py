"""Python binding of libqgemm (ctypes), with the C ABI's names.

Argument marshalling only: torch tensors on the GPU give device pointers,
leading dimensions and the current stream; every step of the computation runs
in the library's HIP kernels.  If ``libqgemm.so`` is missing or cannot be
loaded, importing this module raises -- there is no fallback path.  The int8
attention layer's functions also need ``_qcall.so`` and raise without it.

Layouts follow ``include/qgemm.h``: A ``[M][K]`` row-major, B ``[N][K]``
(column-major K x N), packed int4 operands as ``uint8`` ``[rows][K/2]`` with
element 2i in the low nibble of byte i, per-output-channel int32 bias /
Q31 multiplier / shift, NHWC activations and OHWI weights for the conv.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

# QG_LIB may point the loader at another build of the same library (the
# tests load one built with host-side sanitizers this way)
_LIB_PATH = os.environ.get("QG_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                     "libqgemm.so")

QG_OK = 0
QG_ERR_NULLPTR = 1
QG_ERR_INVALID = 2
QG_ERR_NO_DEVICE = 3
QG_ERR_LAUNCH = 4

QG_S4S4_MAX_K = 131040
QG_W4A8_MAX_K = 131040
QG_S8S8_DEQUANT_MAX_K = 131056

QG_DT_F32 = 0
QG_DT_F16 = 1
QG_DT_BF16 = 2
_QUANT_DTYPES = {torch.float32: QG_DT_F32, torch.float16: QG_DT_F16,
                 torch.bfloat16: QG_DT_BF16}


class QGemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is not built; run __graft_entry__.build() "
                          "(or python conv_qgemm_amd/build.py)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I64, I32, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    lib.qgemm_s8s8_requant.argtypes = [P, I64, P, I64, P, P, P, P, I64, I64, I64, I64, P]
    lib.qgemm_s8s8_requant.restype = S
    lib.qgemm_s4s4_i32.argtypes = [P, I64, P, I64, P, I64, I64, I64, I64, P]
    lib.qgemm_s4s4_i32.restype = S
    lib.qgemm_w4a8_requant.argtypes = [P, I64, P, I64, P, P, P, P, I64, I64, I64, I64, P]
    lib.qgemm_w4a8_requant.restype = S
    lib.qgemm_s4s4_f16.argtypes = [P, I64, P, I64, P, P, P, I64, I64, I64, I64, P]
    lib.qgemm_s4s4_f16.restype = S
    lib.qgemm_w4a8_requant_msb.argtypes = [P, I64, P, I64, P, P, P, P, I64, I64, I64, I64, P]
    lib.qgemm_w4a8_requant_msb.restype = S
    lib.qconv2d_nhwc_s8_requant.argtypes = [P, P, P, P, P, P] + [I32] * 11 + [P]
    lib.qconv2d_nhwc_s8_requant.restype = S
    lib.qdwconv2d_nhwc_s8_requant.argtypes = [P, P, P, P, P, P] + [I32] * 10 + [P]
    lib.qdwconv2d_nhwc_s8_requant.restype = S
    lib.qquant_per_token.argtypes = [P, I32, I64, P, I64, P, I64, I64, ctypes.c_float, I32, P]
    lib.qquant_per_token.restype = S
    Z = ctypes.c_size_t
    lib.qgemm_s8s8_requant_zp_workspace_size.argtypes = [I64, I64]
    lib.qgemm_s8s8_requant_zp_workspace_size.restype = Z
    lib.qgemm_s8s8_requant_zp.argtypes = [P, I64, P, I64, P, P, P, I32, I32, I32, I32, I32, P,
                                          I64, I64, I64, I64, P, Z, P]
    lib.qgemm_s8s8_requant_zp.restype = S
    lib.qgemm_s8s8_requant_zp_noalloc.argtypes = [P, I64, P, I64, P, P, P, I32, I32, I32, I32,
                                                  I32, P, I64, I64, I64, I64, P]
    lib.qgemm_s8s8_requant_zp_noalloc.restype = S
    lib.qconv2d_nhwc_s8_requant_zp_workspace_size.argtypes = [I32] * 10
    lib.qconv2d_nhwc_s8_requant_zp_workspace_size.restype = Z
    lib.qconv2d_nhwc_s8_requant_zp.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, P] + \
        [I32] * 11 + [P, Z, P]
    lib.qconv2d_nhwc_s8_requant_zp.restype = S
    lib.qdwconv2d_nhwc_s8_requant_zp_workspace_size.argtypes = [I32]
    lib.qdwconv2d_nhwc_s8_requant_zp_workspace_size.restype = Z
    lib.qdwconv2d_nhwc_s8_requant_zp.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, P] + \
        [I32] * 10 + [P, Z, P]
    lib.qdwconv2d_nhwc_s8_requant_zp.restype = S
    F = ctypes.c_float
    lib.qgemm_s8s8_dequant.argtypes = [P, I64, P, I64, P, P, P, P, I32, I64, I64, I64, I64, P]
    lib.qgemm_s8s8_dequant.restype = S
    cache, batch = [P, P, P, P, I64, I32, P, I64, I32], [P, P]
    lib.qkv_append_rope.argtypes = [P, I64, P, I64, P, I64, I32, P, I32, I64, I32, P, I64] + \
        cache + batch + [I64] + [I32] * 5 + [P]
    lib.qkv_append_rope.restype = S
    lib.qkv_read.argtypes = cache + batch + [P, P, I32, I64, I32, I32, I32, P]
    lib.qkv_read.restype = S
    lib.qattn_kv8_workspace_size.argtypes = [I64] + [I32] * 6
    lib.qattn_kv8_workspace_size.restype = Z
    lib.qattn_kv8.argtypes = [P, I64, I32] + cache + batch + [F, I32, P, I64, P, I64] + \
        [I32] * 6 + [P, Z, P]
    lib.qattn_kv8.restype = S
    lib.qg_status_string.argtypes = [S]
    lib.qg_status_string.restype = ctypes.c_char_p
    lib.qg_version.argtypes = []
    lib.qg_version.restype = S
    return lib


class _NoCalls:
    """In the place of the module that is missing: the first use says so."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError("conv_qgemm_amd/_qcall.so is not built for this Python and torch; run "
                          "__graft_entry__.build() (or python conv_qgemm_amd/build.py)") from self._why


def _load_calls():
    """The library's calls of one decoding step without ctypes' conversions
    (`lib` has them too).  The int8 attention layer's functions need it, the
    others only `lib`."""
    try:
        from conv_qgemm_amd import _qcall
    except ImportError as e:
        return _NoCalls(e)
    for name in ("qgemm_s8s8_dequant", "qkv_append_rope", "qkv_read", "qattn_kv8_workspace_size",
                 "qattn_kv8"):
        _qcall.bind(name, ctypes.cast(getattr(lib, name), ctypes.c_void_p).value)
    return _qcall


lib = _load()
_calls = _load_calls()
EXPORTS = ("qgemm_s8s8_requant", "qgemm_s4s4_i32", "qgemm_s4s4_f16", "qgemm_w4a8_requant",
           "qgemm_w4a8_requant_msb",
           "qconv2d_nhwc_s8_requant", "qdwconv2d_nhwc_s8_requant", "qquant_per_token",
           "qgemm_s8s8_requant_zp_workspace_size", "qgemm_s8s8_requant_zp",
           "qgemm_s8s8_requant_zp_noalloc",
           "qconv2d_nhwc_s8_requant_zp_workspace_size", "qconv2d_nhwc_s8_requant_zp",
           "qdwconv2d_nhwc_s8_requant_zp_workspace_size", "qdwconv2d_nhwc_s8_requant_zp",
           "qgemm_s8s8_dequant", "qkv_append_rope", "qkv_read", "qattn_kv8_workspace_size",
           "qattn_kv8",
           "qg_status_string", "qg_version")


def status_string(status: int) -> str:
    return lib.qg_status_string(int(status)).decode()


def version() -> int:
    return int(lib.qg_version())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, what: str):
    if status != QG_OK:
        raise QGemmError(status, what)


def _on_device(t, name):
    """The library launches on the current HIP device: every tensor must live
    there (a host or foreign-device pointer would reach the kernels)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor, got one on {t.device}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _mat(t, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    _on_device(t, name)
    return t


def _vec(t, n, name):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.dim() != 1 or t.numel() < n or t.stride(0) != 1:
        raise ValueError(f"{name} must be a contiguous int32 vector of length >= {n}")
    _on_device(t, name)
    return t


def qgemm_s8s8_requant(A, B, bias, mult, shift, C=None, stream=None):
    """C[m][n] = requant(sum_k A[m][k] * B[n][k]); A int8 [M, K], B int8 [N, K]."""
    _mat(A, torch.int8, "A")
    _mat(B, torch.int8, "B")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int8, device=A.device)
    _mat(C, torch.int8, "C")
    st = lib.qgemm_s8s8_requant(_ptr(A), A.stride(0), _ptr(B), B.stride(0),
                                _ptr(_vec(bias, N, "bias")), _ptr(_vec(mult, N, "mult")),
                                _ptr(_vec(shift, N, "shift")), _ptr(C), C.stride(0), M, N, K,
                                _stream(stream))
    _check(st, "qgemm_s8s8_requant")
    return C


def qgemm_s4s4_i32(A, B, C=None, K=None, stream=None):
    """C = A * B^T over packed int4 rows; A uint8 [M, K/2], B uint8 [N, K/2]."""
    _mat(A, torch.uint8, "A")
    _mat(B, torch.uint8, "B")
    M = A.shape[0]
    N = B.shape[0]
    if K is None:
        K = 2 * A.shape[1]
    if 2 * A.shape[1] < K or 2 * B.shape[1] < K:
        raise ValueError("packed rows shorter than K")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int32, device=A.device)
    _mat(C, torch.int32, "C")
    st = lib.qgemm_s4s4_i32(_ptr(A), 2 * A.stride(0), _ptr(B), 2 * B.stride(0), _ptr(C),
                            C.stride(0), M, N, K, _stream(stream))
    _check(st, "qgemm_s4s4_i32")
    return C


def _fvec(t, n, name):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.dim() != 1 or t.numel() < n or t.stride(0) != 1:
        raise ValueError(f"{name} must be a contiguous float32 vector of length >= {n}")
    _on_device(t, name)
    return t


def qgemm_s4s4_f16(A, B, scale_a=None, scale_b=None, C=None, K=None, stream=None):
    """packed int4 A uint8 [M, K/2] x packed int4 B uint8 [N, K/2] -> float16
    C = fp16(fp32(acc) * scale_a[m] * scale_b[n]); the scales are optional
    float32 vectors."""
    _mat(A, torch.uint8, "A")
    _mat(B, torch.uint8, "B")
    M = A.shape[0]
    N = B.shape[0]
    if K is None:
        K = 2 * A.shape[1]
    if 2 * A.shape[1] < K or 2 * B.shape[1] < K:
        raise ValueError("packed rows shorter than K")
    if C is None:
        C = torch.empty((M, N), dtype=torch.float16, device=A.device)
    _mat(C, torch.float16, "C")
    st = lib.qgemm_s4s4_f16(_ptr(A), 2 * A.stride(0), _ptr(B), 2 * B.stride(0),
                            _ptr(_fvec(scale_a, M, "scale_a")), _ptr(_fvec(scale_b, N, "scale_b")),
                            _ptr(C), C.stride(0), M, N, K, _stream(stream))
    _check(st, "qgemm_s4s4_f16")
    return C


def qgemm_w4a8_requant(A, B, bias, mult, shift, C=None, K=None, stream=None, msb_first=False):
    """int8 activations A [M, K] x packed int4 weights B uint8 [N, K/2] -> int8.
    msb_first: the weights hold element 2i in the high nibble of byte i
    (qgemm_w4a8_requant_msb)."""
    _mat(A, torch.int8, "A")
    _mat(B, torch.uint8, "B")
    M = A.shape[0]
    N = B.shape[0]
    if K is None:
        K = A.shape[1]
    if A.shape[1] < K or 2 * B.shape[1] < K:
        raise ValueError("rows shorter than K")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int8, device=A.device)
    _mat(C, torch.int8, "C")
    f = lib.qgemm_w4a8_requant_msb if msb_first else lib.qgemm_w4a8_requant
    st = f(_ptr(A), A.stride(0), _ptr(B), 2 * B.stride(0), _ptr(_vec(bias, N, "bias")),
           _ptr(_vec(mult, N, "mult")), _ptr(_vec(shift, N, "shift")), _ptr(C), C.stride(0), M, N,
           K, _stream(stream))
    _check(st, "qgemm_w4a8_requant_msb" if msb_first else "qgemm_w4a8_requant")
    return C


def conv_out_hw(H, W, KH, KW, stride, pad):
    sh, sw = stride
    ph, pw = pad
    return (H + 2 * ph - KH) // sh + 1, (W + 2 * pw - KW) // sw + 1


def qconv2d_nhwc_s8_requant(X, W, bias, mult, shift, stride=(1, 1), pad=(1, 1), Y=None,
                            stream=None):
    """NHWC int8 conv with zero-point-0 padding and the fused requantize.

    X int8 [batch, H, W, C_in] and W int8 [C_out, KH, KW, C_in], both
    contiguous; returns Y int8 [batch, H_out, W_out, C_out].
    """
    if X.dtype != torch.int8 or W.dtype != torch.int8:
        raise TypeError("X and W must be int8")
    if X.dim() != 4 or W.dim() != 4 or not X.is_contiguous() or not W.is_contiguous():
        raise ValueError("X [B,H,W,C_in] and W [C_out,KH,KW,C_in] must be contiguous 4-D")
    _on_device(X, "X")
    _on_device(W, "W")
    batch, H, Wd, C_in = X.shape
    C_out, KH, KW, C_in2 = W.shape
    if C_in2 != C_in:
        raise ValueError("X and W disagree on C_in")
    Ho, Wo = conv_out_hw(H, Wd, KH, KW, stride, pad)
    if Y is None:
        Y = torch.empty((batch, max(Ho, 0), max(Wo, 0), C_out), dtype=torch.int8,
                        device=X.device)
    if not Y.is_contiguous() or Y.dtype != torch.int8 or tuple(Y.shape) != (batch, Ho, Wo, C_out):
        raise ValueError("Y must be a contiguous int8 [batch, H_out, W_out, C_out] tensor")
    _on_device(Y, "Y")
    st = lib.qconv2d_nhwc_s8_requant(_ptr(X), _ptr(W), _ptr(_vec(bias, C_out, "bias")),
                                     _ptr(_vec(mult, C_out, "mult")),
                                     _ptr(_vec(shift, C_out, "shift")), _ptr(Y),
                                     batch, H, Wd, C_in, C_out, KH, KW, stride[0], stride[1],
                                     pad[0], pad[1], _stream(stream))
    _check(st, "qconv2d_nhwc_s8_requant")
    return Y


def qdwconv2d_nhwc_s8_requant(X, W, bias, mult, shift, stride=(1, 1), pad=(1, 1), Y=None,
                              stream=None):
    """Depthwise NHWC int8 conv (output channel c sees only input channel c)
    with zero-point-0 padding and the fused requantize.

    X int8 [batch, H, W, C] and W int8 [KH, KW, C], both contiguous; returns
    Y int8 [batch, H_out, W_out, C].
    """
    if X.dtype != torch.int8 or W.dtype != torch.int8:
        raise TypeError("X and W must be int8")
    if X.dim() != 4 or W.dim() != 3 or not X.is_contiguous() or not W.is_contiguous():
        raise ValueError("X [B,H,W,C] and W [KH,KW,C] must be contiguous")
    _on_device(X, "X")
    _on_device(W, "W")
    batch, H, Wd, C = X.shape
    KH, KW, C2 = W.shape
    if C2 != C:
        raise ValueError("X and W disagree on C")
    Ho, Wo = conv_out_hw(H, Wd, KH, KW, stride, pad)
    if Y is None:
        Y = torch.empty((batch, max(Ho, 0), max(Wo, 0), C), dtype=torch.int8, device=X.device)
    if not Y.is_contiguous() or Y.dtype != torch.int8 or tuple(Y.shape) != (batch, Ho, Wo, C):
        raise ValueError("Y must be a contiguous int8 [batch, H_out, W_out, C] tensor")
    _on_device(Y, "Y")
    st = lib.qdwconv2d_nhwc_s8_requant(_ptr(X), _ptr(W), _ptr(_vec(bias, C, "bias")),
                                       _ptr(_vec(mult, C, "mult")), _ptr(_vec(shift, C, "shift")),
                                       _ptr(Y), batch, H, Wd, C, KH, KW, stride[0], stride[1],
                                       pad[0], pad[1], _stream(stream))
    _check(st, "qdwconv2d_nhwc_s8_requant")
    return Y


def qquant_per_token(X, bits=8, clip_ratio=1.0, Q=None, scale=None, stream=None):
    """Symmetric per-token quantization of X [M, K] (float32, float16 or
    bfloat16, unit column stride): scale[m] = max|X[m]| / (qmax / clip_ratio),
    codes X / scale rounded half away from zero, clamped to +-qmax (127 for
    bits 8, 7 for bits 4).  Returns (Q, scale): Q int8 [M, K], or for bits 4
    uint8 [M, K/2] with element 2i in the low nibble of byte i; scale float32
    [M]."""
    if X.dtype not in _QUANT_DTYPES:
        raise TypeError(f"X must be float32, float16 or bfloat16, got {X.dtype}")
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D tensor with unit column stride")
    _on_device(X, "X")
    M, K = X.shape
    if bits == 8:
        qdtype, qcols = torch.int8, K
    elif bits == 4:
        qdtype, qcols = torch.uint8, K // 2
    else:
        raise ValueError("bits must be 8 or 4")
    if Q is None:
        Q = torch.empty((M, qcols), dtype=qdtype, device=X.device)
    _mat(Q, qdtype, "Q")
    if Q.shape[0] != M or Q.shape[1] < qcols:
        raise ValueError(f"Q must have {M} rows of at least {qcols} columns")
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=X.device)
    if scale.dtype != torch.float32 or scale.dim() != 1 or scale.numel() < M or \
            scale.stride(0) != 1:
        raise ValueError(f"scale must be a contiguous float32 vector of length >= {M}")
    _on_device(scale, "scale")
    ldq = Q.stride(0) * (2 if bits == 4 else 1)
    st = lib.qquant_per_token(_ptr(X), _QUANT_DTYPES[X.dtype], X.stride(0), _ptr(Q), ldq,
                              _ptr(scale), M, K, float(clip_ratio), bits, _stream(stream))
    _check(st, "qquant_per_token")
    return Q, scale


# ---- asymmetric (zero-point) forms ----

def _workspace(ws, need, device):
    """The caller's workspace (a uint8 GPU tensor of at least `need` bytes),
    or a new one."""
    if need == 0:
        raise ValueError("the library rejects this shape")
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of >= {need} bytes")
    _on_device(ws, "workspace")
    return ws


def qgemm_s8s8_requant_zp(A, B, bias, mult, shift, a_zero, b_zero, out_zero, C=None,
                          workspace=None, stream=None, act=(-128, 127)):
    """Asymmetric int8 GEMM: C = requant(sum_k (A - a_zero)(B - b_zero)) +
    out_zero, saturated to [act[0], act[1]] (the int8 range by default;
    (out_zero, 127) is a fused ReLU).  A int8 [M, K], B int8 [N, K]."""
    _mat(A, torch.int8, "A")
    _mat(B, torch.int8, "B")
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError("A and B disagree on K")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int8, device=A.device)
    _mat(C, torch.int8, "C")
    ws = _workspace(workspace, int(lib.qgemm_s8s8_requant_zp_workspace_size(M, N)), A.device)
    st = lib.qgemm_s8s8_requant_zp(_ptr(A), A.stride(0), _ptr(B), B.stride(0),
                                   _ptr(_vec(bias, N, "bias")), _ptr(_vec(mult, N, "mult")),
                                   _ptr(_vec(shift, N, "shift")), int(a_zero), int(b_zero),
                                   int(out_zero), int(act[0]), int(act[1]), _ptr(C), C.stride(0),
                                   M, N, K, _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "qgemm_s8s8_requant_zp")
    return C


def qgemm_s8s8_requant_zp_noalloc(A, B, bias, mult, shift, a_zero, b_zero, out_zero, C=None,
                                  stream=None, act=(-128, 127)):
    """qgemm_s8s8_requant_zp through the library's allocation-free entry
    point: no workspace, the compensation sums stay in the library's own
    per-GPU array (M + N up to about 262,000; calls that overlap on one GPU
    race on it).  With C given, nothing is allocated on this path."""
    _mat(A, torch.int8, "A")
    _mat(B, torch.int8, "B")
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError("A and B disagree on K")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int8, device=A.device)
    _mat(C, torch.int8, "C")
    st = lib.qgemm_s8s8_requant_zp_noalloc(_ptr(A), A.stride(0), _ptr(B), B.stride(0),
                                           _ptr(_vec(bias, N, "bias")),
                                           _ptr(_vec(mult, N, "mult")),
                                           _ptr(_vec(shift, N, "shift")), int(a_zero),
                                           int(b_zero), int(out_zero), int(act[0]), int(act[1]),
                                           _ptr(C), C.stride(0), M, N, K, _stream(stream))
    _check(st, "qgemm_s8s8_requant_zp_noalloc")
    return C


def qconv2d_nhwc_s8_requant_zp(X, W, bias, mult, shift, a_zero, b_zero, out_zero, stride=(1, 1),
                               pad=(1, 1), Y=None, workspace=None, stream=None, act=(-128, 127)):
    """Asymmetric NHWC int8 conv: padding holds a_zero, products are
    (X - a_zero)(W - b_zero), the output gets out_zero before the
    saturation to [act[0], act[1]].  X [batch, H, W, C_in],
    W [C_out, KH, KW, C_in]."""
    if X.dtype != torch.int8 or W.dtype != torch.int8:
        raise TypeError("X and W must be int8")
    if X.dim() != 4 or W.dim() != 4 or not X.is_contiguous() or not W.is_contiguous():
        raise ValueError("X [B,H,W,C_in] and W [C_out,KH,KW,C_in] must be contiguous 4-D")
    _on_device(X, "X")
    _on_device(W, "W")
    batch, H, Wd, C_in = X.shape
    C_out, KH, KW, C_in2 = W.shape
    if C_in2 != C_in:
        raise ValueError("X and W disagree on C_in")
    Ho, Wo = conv_out_hw(H, Wd, KH, KW, stride, pad)
    if Y is None:
        Y = torch.empty((batch, max(Ho, 0), max(Wo, 0), C_out), dtype=torch.int8,
                        device=X.device)
    if not Y.is_contiguous() or Y.dtype != torch.int8 or tuple(Y.shape) != (batch, Ho, Wo, C_out):
        raise ValueError("Y must be a contiguous int8 [batch, H_out, W_out, C_out] tensor")
    _on_device(Y, "Y")
    need = int(lib.qconv2d_nhwc_s8_requant_zp_workspace_size(batch, H, Wd, C_out, KH, KW,
                                                             stride[0], stride[1], pad[0],
                                                             pad[1]))
    ws = _workspace(workspace, need, X.device)
    st = lib.qconv2d_nhwc_s8_requant_zp(_ptr(X), _ptr(W), _ptr(_vec(bias, C_out, "bias")),
                                        _ptr(_vec(mult, C_out, "mult")),
                                        _ptr(_vec(shift, C_out, "shift")), int(a_zero),
                                        int(b_zero), int(out_zero), int(act[0]), int(act[1]),
                                        _ptr(Y), batch, H, Wd, C_in,
                                        C_out, KH, KW, stride[0], stride[1], pad[0], pad[1],
                                        _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "qconv2d_nhwc_s8_requant_zp")
    return Y


def qdwconv2d_nhwc_s8_requant_zp(X, W, bias, mult, shift, a_zero, b_zero, out_zero,
                                 stride=(1, 1), pad=(1, 1), Y=None, workspace=None, stream=None,
                                 act=(-128, 127)):
    """Asymmetric depthwise NHWC int8 conv (W [KH, KW, C]); zero points as
    for qconv2d_nhwc_s8_requant_zp."""
    if X.dtype != torch.int8 or W.dtype != torch.int8:
        raise TypeError("X and W must be int8")
    if X.dim() != 4 or W.dim() != 3 or not X.is_contiguous() or not W.is_contiguous():
        raise ValueError("X [B,H,W,C] and W [KH,KW,C] must be contiguous")
    _on_device(X, "X")
    _on_device(W, "W")
    batch, H, Wd, C = X.shape
    KH, KW, C2 = W.shape
    if C2 != C:
        raise ValueError("X and W disagree on C")
    Ho, Wo = conv_out_hw(H, Wd, KH, KW, stride, pad)
    if Y is None:
        Y = torch.empty((batch, max(Ho, 0), max(Wo, 0), C), dtype=torch.int8, device=X.device)
    if not Y.is_contiguous() or Y.dtype != torch.int8 or tuple(Y.shape) != (batch, Ho, Wo, C):
        raise ValueError("Y must be a contiguous int8 [batch, H_out, W_out, C] tensor")
    _on_device(Y, "Y")
    ws = _workspace(workspace, int(lib.qdwconv2d_nhwc_s8_requant_zp_workspace_size(C)), X.device)
    st = lib.qdwconv2d_nhwc_s8_requant_zp(_ptr(X), _ptr(W), _ptr(_vec(bias, C, "bias")),
                                          _ptr(_vec(mult, C, "mult")),
                                          _ptr(_vec(shift, C, "shift")), int(a_zero),
                                          int(b_zero), int(out_zero), int(act[0]), int(act[1]),
                                          _ptr(Y), batch, H, Wd, C,
                                          KH, KW, stride[0], stride[1], pad[0], pad[1],
                                          _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "qdwconv2d_nhwc_s8_requant_zp")
    return Y


# ---- int8 attention layer: float-output GEMM, key/value cache, attention ----
#
# A decoding step makes these calls with little work behind each, so their
# tensors are checked by _calls; the functions that name what is wrong run only
# when a check says no.

_I8, _I32, _F32 = torch.int8, torch.int32, torch.float32


def _ld(t):
    """The row stride of a matrix; a single row's may be anything in torch."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _queue(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _empty(like, dtype, stream, *shape):
    """A new tensor of the stream that the call runs on, so that its memory is
    neither still in use on another stream nor given away before the call ends."""
    if stream is None:
        return _calls.empty(like, dtype, *shape)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return _calls.empty(like, dtype, *shape)


def _float_vec(t, n, name, dev):
    if t is None:
        return None
    at = _calls.vector(t, _F32, n, dev)
    if at is False:
        _fvec(t, n, name)
        raise ValueError(f"{name} must be a float32 vector on the operands' device")
    return at


def qgemm_s8s8_dequant(A, B, scale_a=None, scale_b=None, bias=None, dtype=torch.bfloat16, C=None,
                       stream=None):
    """C[m][n] = dtype(fp32(sum_k A[m][k] * B[n][k]) * scale_a[m] * scale_b[n]
    + bias[n]); A int8 [M, K] (the codes of qquant_per_token, scale_a its
    scales), B int8 [N, K] with a scale for each row; the float32 vectors
    scale_a, scale_b and bias are optional.  dtype float32, float16 or
    bfloat16."""
    args = _calls.operands(A, B)
    if args is None:
        _mat(A, torch.int8, "A")
        _mat(B, torch.int8, "B")
        raise ValueError("A and B disagree on K")
    dev, a, lda, b, ldb, M, N, K = args
    if C is None:
        code = _QUANT_DTYPES.get(dtype)
        if code is None:
            raise TypeError(f"C must be float32, float16 or bfloat16, got {dtype}")
        C = _empty(A, dtype, stream, M, N)
        ldc = N
    else:
        code = _QUANT_DTYPES.get(C.dtype)
        if code is None:
            raise TypeError(f"C must be float32, float16 or bfloat16, got {C.dtype}")
        _mat(C, C.dtype, "C")
        if C.shape[0] != M or C.shape[1] != N:
            raise ValueError(f"C must be [{M}, {N}]")
        ldc = _ld(C)
    st = _calls.qgemm_s8s8_dequant(a, lda, b, ldb, _float_vec(scale_a, M, "scale_a", dev),
                                   _float_vec(scale_b, N, "scale_b", dev),
                                   _float_vec(bias, N, "bias", dev), C.data_ptr(), code, ldc, M, N,
                                   K, _queue(stream, dev))
    if st:
        _check(st, "qgemm_s8s8_dequant")
    return C


class KVCache(NamedTuple):
    """A paged int8 key/value cache: codes ``k`` and ``v`` int8 [blocks, heads,
    block_size, head_dim], scales ``k_scale`` and ``v_scale`` float32 [blocks,
    heads]; a code c of block b and head h stands for c * scale[b, h]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv_cache(num_blocks, heads, block_size, head_dim, device="cuda"):
    """An empty KVCache (block_size 16, 32, 64 or 128; head_dim 64, 128 or 256)."""
    def codes():
        return torch.zeros(num_blocks, heads, block_size, head_dim, dtype=torch.int8, device=device)

    def scales():
        return torch.zeros(num_blocks, heads, dtype=torch.float32, device=device)

    return KVCache(codes(), codes(), scales(), scales())


def _refuse_cache(cache, table):
    for t, name in ((cache.k, "cache.k"), (cache.v, "cache.v")):
        if t.dtype != torch.int8 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int8 [blocks, heads, block_size, "
                             "head_dim] tensor")
        _on_device(t, name)
    if cache.v.shape != cache.k.shape:
        raise ValueError("cache.k and cache.v disagree on their shape")
    for t, name in ((cache.k_scale, "cache.k_scale"), (cache.v_scale, "cache.v_scale")):
        if t.dtype != torch.float32 or t.shape != cache.k.shape[:2] or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 {list(cache.k.shape[:2])} tensor")
        _on_device(t, name)
    if table.dim() == 2 and table.shape[1] == 1:
        table = table.contiguous()
    _mat(table, torch.int32, "block_table")
    raise ValueError("cache must be a KVCache")


def _cache_args(cache, table):
    """The cache's part of the argument list, its shape and its device."""
    args = _calls.cache_args(cache, table)
    if args is None:
        _refuse_cache(cache, table)
    return args


def _lens(t, n, name, dev):
    at = _calls.vector(t, _I32, n, dev)
    if at is False or t.shape[0] != n:
        if t.dtype == torch.int32 and t.dim() == 1 and t.numel() == n and t.is_contiguous():
            _on_device(t, name)
        raise ValueError(f"{name} must be a contiguous int32 vector of length {n}")
    return at


def _rows(t, tokens, heads, D, dtype, name, dev):
    """[tokens, heads, D] of dtype with dense heads; the row stride in elements."""
    ld = _calls.rows(t, tokens, heads, D, dtype, dev)
    if ld is None:
        if t.dim() == 3 and tuple(t.shape) == (tokens, heads, D) and t.stride(2) == 1 and \
                (heads == 1 or t.stride(1) == D):
            if t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            _on_device(t, name)
        raise ValueError(f"{name} must be [{tokens}, {heads}, {D}] with dense heads")
    return ld


def qkv_append_rope(q, k, v, cache, block_table, cu_seqlens, kv_lens, max_q, cos_sin=None,
                    interleaved=False, q_out=None, stream=None):
    """Rotates new queries and keys by their positions and writes the new keys
    and values, coded to int8, into the cache (in place).  Returns the rotated
    queries (None when q is None).

    q [tokens, q_heads, D], k and v [tokens, heads, D] (float32, float16 or
    bfloat16; slices of one fused projection will do); cos_sin float32
    [positions, rot_dim], cosines then sines; block_table int32 [seqs,
    columns]; cu_seqlens int32 [seqs + 1] and kv_lens int32 [seqs] as for
    qattn_kv8.  Rotation pairs element i with i + rot_dim / 2, or, interleaved,
    2i with 2i + 1."""
    args, heads, D, dev = _cache_args(cache, block_table)
    dtype = k.dtype
    code = _QUANT_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"k must be float32, float16 or bfloat16, got {dtype}")
    tokens, seqs = k.shape[0], block_table.shape[0]
    ldk = _rows(k, tokens, heads, D, dtype, "k", dev)
    ldv = _rows(v, tokens, heads, D, dtype, "v", dev)
    qp = op = None
    ldq = ldqo = 0
    q_heads = heads
    if q is not None:
        q_heads = q.shape[1]
        ldq = _rows(q, tokens, q_heads, D, dtype, "q", dev)
        if q_out is None:
            q_out = _empty(q, dtype, stream, tokens, q_heads, D)
            ldqo = q_heads * D
        else:
            ldqo = _rows(q_out, tokens, q_heads, D, dtype, "q_out", dev)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    table, npos, rot = None, 0, 0
    if cos_sin is not None:
        found = _calls.table(cos_sin, dev)
        if found is None:
            _mat(cos_sin, torch.float32, "cos_sin")
            raise ValueError("cos_sin must be contiguous")
        table, npos, rot = found
    cu, lens = _lens(cu_seqlens, seqs + 1, "cu_seqlens", dev), _lens(kv_lens, seqs, "kv_lens", dev)
    if tokens == 0:  # empty tensors have no address
        return q_out
    st = _calls.qkv_append_rope(qp, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, code, table, rot,
                                npos, 1 if interleaved else 0, op, ldqo, *args, cu, lens, tokens,
                                seqs, max_q, q_heads, heads, D, _queue(stream, dev))
    if st:
        _check(st, "qkv_append_rope")
    return q_out


def qkv_read(cache, block_table, start, cu_out, tokens, dtype=torch.bfloat16, stream=None):
    """Cached tokens start[b] .. of each sequence b (cu_out[b + 1] - cu_out[b]
    of them) back as values: (k, v), each [tokens, heads, D] of dtype, one
    sequence after the other; `tokens` is cu_out's last entry."""
    args, heads, D, dev = _cache_args(cache, block_table)
    code = _QUANT_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    seqs = block_table.shape[0]
    first, cu = _lens(start, seqs, "start", dev), _lens(cu_out, seqs + 1, "cu_out", dev)
    k = _empty(cache.k, dtype, stream, tokens, heads, D)
    v = _empty(cache.k, dtype, stream, tokens, heads, D)
    if tokens:
        st = _calls.qkv_read(*args, first, cu, k.data_ptr(), v.data_ptr(), code, tokens, seqs, heads,
                          D, _queue(stream, dev))
        if st:
            _check(st, "qkv_read")
    return k, v


def qattn_kv8(q, cache, block_table, cu_seqlens, kv_lens, max_q, max_kv, scale=None, causal=True,
              out=None, return_lse=False, workspace=None, stream=None):
    """Attention of new queries over the paged int8 cache, whose last tokens
    are the new ones.  q [tokens, q_heads, D] float16 or bfloat16, the
    sequences one after the other; cu_seqlens int32 [seqs + 1] their running
    sums, kv_lens int32 [seqs] the cached tokens of each with the new ones;
    max_q and max_kv bound the new and the cached tokens of any sequence.
    Query head h reads cache head h // (q_heads // heads); scale defaults to
    D ** -0.5.  causal: new token i of n sees the cache up to itself.  Returns
    out [tokens, q_heads, D], or (out, lse float32 [tokens, q_heads]); a query
    that sees nothing gives 0 and -infinity."""
    args, heads, D, dev = _cache_args(cache, block_table)
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"q must be float16 or bfloat16, got {dtype}")
    if q.dim() != 3:
        raise ValueError("q must be [tokens, q_heads, D]")
    tokens, q_heads, _ = q.shape
    seqs = block_table.shape[0]
    ldq = _rows(q, tokens, q_heads, D, dtype, "q", dev)
    if out is None:
        out = _empty(q, dtype, stream, tokens, q_heads, D)
        ldo = q_heads * D
    else:
        ldo = _rows(out, tokens, q_heads, D, dtype, "out", dev)
    cu, lens = _lens(cu_seqlens, seqs + 1, "cu_seqlens", dev), _lens(kv_lens, seqs, "kv_lens", dev)
    lse = _empty(q, _F32, stream, tokens, q_heads) if return_lse else None
    if tokens:
        need = _calls.qattn_kv8_workspace_size(tokens, seqs, max_q, max_kv, q_heads, heads, D)
        ws = None
        if need:
            ws = _workspace(workspace, need, q.device) if workspace is not None else \
                _empty(q, torch.uint8, stream, need)
        st = _calls.qattn_kv8(q.data_ptr(), ldq, _QUANT_DTYPES[dtype], *args, cu, lens,
                           D ** -0.5 if scale is None else scale, 1 if causal else 0,
                           out.data_ptr(), ldo, None if lse is None else lse.data_ptr(), tokens,
                           seqs, max_q, max_kv, q_heads, heads, D,
                           None if ws is None else ws.data_ptr(), need, _queue(stream, dev))
        if st:
            _check(st, "qattn_kv8")
    return (out, lse) if return_lse else out
