"""Thin Python binding of libs3r.so (include/s3r.h).

The functions named ``s3r_*`` mirror the C entry points one to one: they only
marshal torch tensors (device memory) and the current HIP stream into the C
call.  Every step of the computation runs in the library's HIP kernels; if the
library is missing, loading it raises (there is no fallback).

The helpers without the prefix (``quantize``, ``backward_dx``, ``backward_dw``,
``forward_operand``) allocate outputs and workspaces with torch and then call
the entry points.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass, field

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libs3r.so")

S3R_OK = 0
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported combination", -3: "workspace too small",
          -4: "device is not gfx950", -5: "HIP error"}
S3R_F32, S3R_BF16, S3R_I32_RAW, S3R_F32_ACC = 0, 1, 2, 3
RTNE, SR, S3R, S3R_BCAST = 0, 1, 2, 3
EC_NONE, EC_DX_ONLY, EC_TWO_WAY, EC_DW_ONLY = 0, 1, 2, 3
PER_TENSOR, PER_TOKEN = 0, 1
SOFTMAX, SIGMOID = 0, 1
FLAG_NONFINITE, FLAG_TINY_STEP, FLAG_BAD_GROUPS = 1, 2, 8
S3R_NOALLOC_SCRATCH_BYTES = 32 << 20    # include/s3r.h: the no-alloc quantizer's device array

EXPORTED = ["s3r_quantize_workspace", "s3r_quantize", "s3r_quantize_with_amax", "s3r_quantize_noalloc", "s3r_backward_dx",
            "s3r_backward_dw", "s3r_backward_dw_pair", "s3r_backward_dw_pair_workspace", "s3r_backward_workspace", "s3r_swiglu_backward", "s3r_swiglu_amax_workspace",
            "s3r_swiglu_backward_amax", "s3r_swiglu_quantize_workspace", "s3r_swiglu_quantize", "s3r_grouped_workspace", "s3r_grouped_quantize",
            "s3r_grouped_backward_dx", "s3r_grouped_backward_dw", "s3r_mx_workspace", "s3r_mx_operand_workspace",
            "s3r_mx_operand", "s3r_mx_quantize", "s3r_mx_backward_dx", "s3r_mx_backward_dw", "s3r_route_workspace", "s3r_route",
            "s3r_route_backward", "s3r_dispatch", "s3r_combine", "s3r_combine_backward", "s3r_mx_rows",
            "s3r_mx_product", "s3r_mx_linear_workspace", "s3r_mx_linear", "s3r_int_rows", "s3r_int_colsum", "s3r_int_product",
            "s3r_int_linear_workspace", "s3r_int_linear", "s3r_orthogonalize_workspace", "s3r_orthogonalize",
            "s3r_time_next_gemm",
            "s3r_status_string", "s3r_version"]


class S3RError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({code})")
        self.code = code


class QDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("rows_per_example", ctypes.c_int64),
                ("mode", ctypes.c_int32), ("ec", ctypes.c_int32), ("scale", ctypes.c_int32),
                ("layer_id", ctypes.c_uint32), ("seed", ctypes.c_uint64), ("stream", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class RouteDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("keep", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("score", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_uint32)]


def route_desc(tokens, experts, top_k, *, score=SOFTMAX, groups=1, keep=1, group_top=1, renorm=True,
               scale=1.0) -> RouteDesc:
    return RouteDesc(tokens, experts, top_k, groups, keep, group_top, score, 1 if renorm else 0, scale, 0)


class MxPDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("depth", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("ld_b", ctypes.c_int64), ("ld_bs", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("bs_stride", ctypes.c_int64), ("out_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_uint32)]


class IntPDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("depth", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("ld_b", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_uint32)]


class OrthDesc(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("g_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("keep", ctypes.c_float), ("reserved", ctypes.c_uint32)]


def qdesc(rows, cols, rows_per_example=None, mode=S3R, ec=EC_NONE, scale=PER_TENSOR, layer_id=0, seed=0,
          stream=0) -> QDesc:
    S = rows_per_example if rows_per_example is not None else max(rows, 1)
    return QDesc(rows, cols, S, mode, ec, scale, layer_id, seed, stream, 0)


_lib = None


def lib() -> ctypes.CDLL:
    """Load libs3r.so (built in-tree by ``python -m stochastic_rounding_quantization_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run python -m stochastic_rounding_quantization_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    DP = ctypes.POINTER(QDesc)
    L.s3r_quantize_workspace.argtypes = [DP]
    L.s3r_quantize_workspace.restype = SZ
    L.s3r_quantize.argtypes = [DP, P, I32, I64, P, P, P, I64, P, P, P, P, P, P, P, SZ, P]
    L.s3r_quantize.restype = ctypes.c_int
    L.s3r_quantize_with_amax.argtypes = [DP, P, I32, I64, P, P, P, P, I64, P, P, P, P, P, P, SZ, P]
    L.s3r_quantize_with_amax.restype = ctypes.c_int
    L.s3r_quantize_noalloc.argtypes = [DP, P, I32, I64, P, P, P, I64, P, P, P, P, P, P, P]
    L.s3r_quantize_noalloc.restype = ctypes.c_int
    L.s3r_backward_dx.argtypes = [DP, P, I64, P, P, I64, I64, P, P, P, P, P, P, I32, I64, P, SZ, P]
    L.s3r_backward_dx.restype = ctypes.c_int
    L.s3r_backward_dw.argtypes = [DP, P, I64, P, P, I64, I64, P, P, P, P, P, P, I32, I64, P, SZ, P]
    L.s3r_backward_dw.restype = ctypes.c_int
    L.s3r_backward_dw_pair.argtypes = [DP, P, P, I64, P, P, P, I64, I64, P, P, P, P, P, P, P, P, P, P, P, I32, I64,
                                       P, SZ, P]
    L.s3r_backward_dw_pair.restype = ctypes.c_int
    L.s3r_backward_dw_pair_workspace.argtypes = [DP, I64]
    L.s3r_backward_dw_pair_workspace.restype = SZ
    L.s3r_backward_workspace.argtypes = [DP, I64]
    L.s3r_backward_workspace.restype = SZ
    L.s3r_swiglu_backward.argtypes = [I64, I64, P, I64, P, P, I64, P, P, I64, P]
    L.s3r_swiglu_backward.restype = ctypes.c_int
    L.s3r_swiglu_amax_workspace.argtypes = [I64, I64]
    L.s3r_swiglu_amax_workspace.restype = SZ
    L.s3r_swiglu_backward_amax.argtypes = [I64, I64, P, I64, P, P, I64, P, P, I64, P, P, P, P, P, SZ, P]
    L.s3r_swiglu_backward_amax.restype = ctypes.c_int
    L.s3r_swiglu_quantize_workspace.argtypes = [DP]
    L.s3r_swiglu_quantize_workspace.restype = SZ
    L.s3r_swiglu_quantize.argtypes = [DP, DP, P, I64, P, P, I64, P, P, P, P, P, I64, P, P, P, P, P, P, P, P, P, P, SZ,
                                      P]
    L.s3r_swiglu_quantize.restype = ctypes.c_int
    L.s3r_grouped_workspace.argtypes = [DP, I64, I64]
    L.s3r_grouped_workspace.restype = SZ
    L.s3r_grouped_quantize.argtypes = [DP, I64, P, P, I32, I64, P, P, P, I64, P, P, P, P, P, P, P, SZ, P]
    L.s3r_grouped_quantize.restype = ctypes.c_int
    L.s3r_grouped_backward_dx.argtypes = [DP, I64, P, P, I64, P, P, I64, I64, I64, P, P, P, P, P, P, I32, I64, P, P,
                                          SZ, P]
    L.s3r_grouped_backward_dx.restype = ctypes.c_int
    L.s3r_grouped_backward_dw.argtypes = [DP, I64, P, P, I64, P, P, I64, I64, P, P, P, P, P, P, I32, I64, I64, P, P,
                                          SZ, P]
    L.s3r_grouped_backward_dw.restype = ctypes.c_int
    L.s3r_mx_workspace.argtypes = [DP, I64]
    L.s3r_mx_workspace.restype = SZ
    L.s3r_mx_operand_workspace.argtypes = [I64, I64]
    L.s3r_mx_operand_workspace.restype = SZ
    L.s3r_mx_operand.argtypes = [I64, I64, I64, P, I32, I64, P, I64, P, I64, P, P, P, SZ, P]
    L.s3r_mx_quantize.argtypes = [DP, P, I32, I64, P, I64, P, I64, P, I64, P, I64, P, P, P, P, P, P, P, P, SZ, P]
    L.s3r_mx_backward_dx.argtypes = [DP, P, I64, P, I64, P, I64, P, I64, I64, P, P, P, P, P, I64, P, SZ, P]
    L.s3r_mx_backward_dw.argtypes = [DP, P, I64, P, I64, P, I64, P, I64, I64, P, P, P, P, P, I64, P, SZ, P]
    RP, MP = ctypes.POINTER(RouteDesc), ctypes.POINTER(MxPDesc)
    L.s3r_route_workspace.argtypes = [RP]
    L.s3r_route_workspace.restype = SZ
    L.s3r_route.argtypes = [RP, P, I32, I64, P, P, P, P, P, P, P, SZ, P]
    L.s3r_route_backward.argtypes = [RP, P, I32, I64, P, P, P, I64, P]
    L.s3r_dispatch.argtypes = [I64, I64, I64, I64, I32, P, I64, P, P, I64, P]
    L.s3r_combine.argtypes = [I64, I64, I64, I64, I32, P, I64, P, P, P, I64, P]
    L.s3r_combine_backward.argtypes = [I64, I64, I64, I64, I32, P, I64, P, P, P, P, I64, P, P]
    L.s3r_mx_rows.argtypes = [I64, I64, I64, P, P, I32, I64, I64, I64, P, I64, P, I64, I64, P, I64, I64, P, P]
    L.s3r_mx_product.argtypes = [MP, P, I64, P, I64, P, P, P, P, I64, P, P]
    L.s3r_mx_linear_workspace.argtypes = [I64, I64]
    L.s3r_mx_linear_workspace.restype = SZ
    L.s3r_mx_linear.argtypes = [MP, P, P, I32, I64, I64, P, I64, P, P, P, P, I64, P, P, SZ, P]
    IP = ctypes.POINTER(IntPDesc)
    L.s3r_int_rows.argtypes = [I64, I64, I64, P, P, I32, I64, I64, I64, P, I64, P, I64, I64, P, P, P]
    L.s3r_int_colsum.argtypes = [I64, P, I64, I64, P, I64, P, P, P]
    L.s3r_int_product.argtypes = [IP, P, I64, P, P, P, P, P, P, I64, P, P]
    L.s3r_int_linear_workspace.argtypes = [I64, I64]
    L.s3r_int_linear_workspace.restype = SZ
    L.s3r_int_linear.argtypes = [IP, P, P, I32, I64, I64, P, I64, P, P, P, P, P, I64, P, P, SZ, P]
    OP = ctypes.POINTER(OrthDesc)
    L.s3r_orthogonalize_workspace.argtypes = [OP]
    L.s3r_orthogonalize_workspace.restype = SZ
    L.s3r_orthogonalize.argtypes = [OP, P, I64, I64, P, I64, I64, P, SZ, P]
    for f in ("s3r_int_rows", "s3r_int_colsum", "s3r_int_product", "s3r_int_linear", "s3r_orthogonalize"):
        getattr(L, f).restype = ctypes.c_int
    for f in ("s3r_route", "s3r_route_backward", "s3r_dispatch", "s3r_combine", "s3r_combine_backward",
              "s3r_mx_rows", "s3r_mx_product", "s3r_mx_linear"):
        getattr(L, f).restype = ctypes.c_int
    L.s3r_time_next_gemm.argtypes = [P, P]
    L.s3r_time_next_gemm.restype = ctypes.c_int
    L.s3r_status_string.argtypes = [ctypes.c_int]
    L.s3r_status_string.restype = ctypes.c_char_p
    L.s3r_version.argtypes = []
    L.s3r_version.restype = ctypes.c_int
    _lib = L
    return L


# ------------------------------------------------------------ marshalling ----

def _ptr(t):
    return None if t is None else t.data_ptr()      # the argument's declared type makes it a pointer


def _ld(t, default=0):
    if t is None:
        return default
    s = t.stride()
    if len(s) != 2 or s[1] != 1:
        raise ValueError("expected a row-major 2-D tensor (unit column stride)")
    return s[0]


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    # the current stream's handle without a Stream object around it (2 us of a call's 10)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _check(fn, rc):
    if rc != S3R_OK:
        raise S3RError(fn, rc)


def _gdtype(t):
    import torch
    dt = t.dtype
    if dt is torch.float32:
        return S3R_F32
    if dt is torch.bfloat16:
        return S3R_BF16
    raise ValueError(f"unsupported gradient dtype {t.dtype}")


def _odtype(t, accumulate=False):
    import torch
    if t.dtype == torch.float32:
        return S3R_F32_ACC if accumulate else S3R_F32
    if t.dtype == torch.int32:
        return S3R_I32_RAW
    raise ValueError(f"unsupported output dtype {t.dtype}")


def s3r_quantize_workspace(desc: QDesc) -> int:
    return lib().s3r_quantize_workspace(ctypes.byref(desc))


def s3r_quantize(desc: QDesc, G, row_scale, col_scale, Q, delta, code_colsum=None, ec_row=None, ec_col=None,
                 ec_mean=None, flags=None, ws=None, stream=None, *, rc_only=False):
    rc = lib().s3r_quantize(ctypes.byref(desc), _ptr(G), _gdtype(G) if G is not None else S3R_F32,
                            _ld(G, desc.cols), _ptr(row_scale), _ptr(col_scale), _ptr(Q), _ld(Q, desc.cols),
                            _ptr(delta), _ptr(code_colsum), _ptr(ec_row), _ptr(ec_col), _ptr(ec_mean),
                            _ptr(flags), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                            _stream(stream))
    if rc_only:
        return rc
    _check("s3r_quantize", rc)


def s3r_quantize_noalloc(desc: QDesc, G, row_scale, col_scale, Q, delta, code_colsum=None, ec_row=None, ec_col=None,
                         ec_mean=None, flags=None, stream=None, *, rc_only=False):
    rc = lib().s3r_quantize_noalloc(ctypes.byref(desc), _ptr(G), _gdtype(G) if G is not None else S3R_F32,
                                    _ld(G, desc.cols), _ptr(row_scale), _ptr(col_scale), _ptr(Q), _ld(Q, desc.cols),
                                    _ptr(delta), _ptr(code_colsum), _ptr(ec_row), _ptr(ec_col), _ptr(ec_mean),
                                    _ptr(flags), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_quantize_noalloc", rc)


def s3r_quantize_with_amax(desc: QDesc, G, row_scale, col_scale, amax_bits, Q, delta, ec_row=None, ec_col=None,
                           ec_mean=None, flags=None, ws=None, stream=None, *, rc_only=False):
    rc = lib().s3r_quantize_with_amax(ctypes.byref(desc), _ptr(G), _gdtype(G) if G is not None else S3R_F32,
                                      _ld(G, desc.cols), _ptr(row_scale), _ptr(col_scale), _ptr(amax_bits), _ptr(Q),
                                      _ld(Q, desc.cols), _ptr(delta), _ptr(ec_row), _ptr(ec_col), _ptr(ec_mean),
                                      _ptr(flags), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                      _stream(stream))
    if rc_only:
        return rc
    _check("s3r_quantize_with_amax", rc)


def s3r_backward_workspace(desc: QDesc, d_in: int) -> int:
    return lib().s3r_backward_workspace(ctypes.byref(desc), d_in)


def s3r_backward_dx(desc: QDesc, Q, delta, Wq, s_x, r_W, ec_row, ec_col, ec_mean, dX, ws=None, stream=None,
                    *, accumulate=False, rc_only=False):
    d_in = dX.shape[1]
    rc = lib().s3r_backward_dx(ctypes.byref(desc), _ptr(Q), _ld(Q, desc.cols), _ptr(delta), _ptr(Wq),
                               _ld(Wq, d_in), d_in, _ptr(s_x), _ptr(r_W), _ptr(ec_row), _ptr(ec_col),
                               _ptr(ec_mean), _ptr(dX), _odtype(dX, accumulate), _ld(dX, d_in), _ptr(ws),
                               0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_backward_dx", rc)


def s3r_backward_dw(desc: QDesc, Q, delta, Xq, s_w, xs_b, ec_row, ec_col, ec_mean, dW, ws=None, stream=None,
                    *, rc_only=False):
    d_in = dW.shape[1]
    rc = lib().s3r_backward_dw(ctypes.byref(desc), _ptr(Q), _ld(Q, desc.cols), _ptr(delta), _ptr(Xq),
                               _ld(Xq, d_in), d_in, _ptr(s_w), _ptr(xs_b), _ptr(ec_row), _ptr(ec_col),
                               _ptr(ec_mean), _ptr(dW), _odtype(dW), _ld(dW, d_in), _ptr(ws),
                               0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_backward_dw", rc)


def s3r_backward_dw_pair_workspace(desc: QDesc, d_in: int) -> int:
    return lib().s3r_backward_dw_pair_workspace(ctypes.byref(desc), d_in)


def s3r_backward_dw_pair(desc: QDesc, Q0, Q1, delta0, delta1, Xq, s_w0, s_w1, xs_b, ec0, ec1, dW0, dW1, ws=None,
                         stream=None, *, rc_only=False):
    """Both dW products of two projections of one input in one launch; ec0 / ec1 are the
    (ec_row, ec_col, ec_mean) triples of the two quantize calls."""
    d_in = dW0.shape[1]
    if _ld(Q1, desc.cols) != _ld(Q0, desc.cols) or _ld(dW1, d_in) != _ld(dW0, d_in) or dW1.dtype != dW0.dtype:
        raise ValueError("the two products need codes and outputs of one layout")
    rc = lib().s3r_backward_dw_pair(
        ctypes.byref(desc), _ptr(Q0), _ptr(Q1), _ld(Q0, desc.cols), _ptr(delta0), _ptr(delta1), _ptr(Xq),
        _ld(Xq, d_in), d_in, _ptr(s_w0), _ptr(s_w1), _ptr(xs_b), _ptr(ec0[0]), _ptr(ec0[1]), _ptr(ec0[2]),
        _ptr(ec1[0]), _ptr(ec1[1]), _ptr(ec1[2]), _ptr(dW0), _ptr(dW1), _odtype(dW0), _ld(dW0, d_in), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_backward_dw_pair", rc)


def s3r_swiglu_backward(dH, A_gate, A_up, G_gate, G_up, stream=None, *, rc_only=False):
    """bf16 tensors are passed as torch.bfloat16 (their bit patterns are the C ABI's uint16)."""
    T, F = dH.shape
    if A_up.stride() != A_gate.stride() or G_up.stride() != G_gate.stride():
        raise ValueError("A_gate / A_up and G_gate / G_up must share their layouts")
    rc = lib().s3r_swiglu_backward(T, F, _ptr(dH), _ld(dH, F), _ptr(A_gate), _ptr(A_up), _ld(A_gate, F),
                                   _ptr(G_gate), _ptr(G_up), _ld(G_gate, F), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_swiglu_backward", rc)


def s3r_swiglu_amax_workspace(T: int, F: int) -> int:
    return lib().s3r_swiglu_amax_workspace(T, F)


def s3r_swiglu_backward_amax(dH, A_gate, A_up, G_gate, G_up, row_scale, col_scale_gate, col_scale_up, amax_bits,
                             ws, stream=None, *, rc_only=False):
    """Glue and the gate / up amax (uint32 [2] device tensor amax_bits) in one pass."""
    T, F = dH.shape
    if A_up.stride() != A_gate.stride() or G_up.stride() != G_gate.stride():
        raise ValueError("A_gate / A_up and G_gate / G_up must share their layouts")
    rc = lib().s3r_swiglu_backward_amax(T, F, _ptr(dH), _ld(dH, F), _ptr(A_gate), _ptr(A_up), _ld(A_gate, F),
                                        _ptr(G_gate), _ptr(G_up), _ld(G_gate, F), _ptr(row_scale),
                                        _ptr(col_scale_gate), _ptr(col_scale_up), _ptr(amax_bits), _ptr(ws),
                                        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_swiglu_backward_amax", rc)


def s3r_swiglu_quantize_workspace(desc: QDesc) -> int:
    return lib().s3r_swiglu_quantize_workspace(ctypes.byref(desc))


def s3r_swiglu_quantize(desc_gate: QDesc, desc_up: QDesc, dH, A_gate, A_up, row_scale, col_scale_gate, col_scale_up,
                        Q_gate, Q_up, delta_gate, delta_up, ec_gate=(None, None, None), ec_up=(None, None, None),
                        flags=None, ws=None, stream=None, *, rc_only=False):
    """The gate and up quantizers with the glue inside (G_gate, G_up never written); ec_gate / ec_up are
    (ec_row, ec_col, ec_mean) triples."""
    F = desc_gate.cols
    if A_up.stride() != A_gate.stride() or _ld(Q_up, F) != _ld(Q_gate, F):
        raise ValueError("A_gate / A_up and Q_gate / Q_up must share their layouts")
    rc = lib().s3r_swiglu_quantize(
        ctypes.byref(desc_gate), ctypes.byref(desc_up), _ptr(dH), _ld(dH, F), _ptr(A_gate), _ptr(A_up),
        _ld(A_gate, F), _ptr(row_scale), _ptr(col_scale_gate), _ptr(col_scale_up), _ptr(Q_gate), _ptr(Q_up),
        _ld(Q_gate, F), _ptr(delta_gate), _ptr(delta_up), _ptr(ec_gate[0]), _ptr(ec_gate[1]), _ptr(ec_gate[2]),
        _ptr(ec_up[0]), _ptr(ec_up[1]), _ptr(ec_up[2]), _ptr(flags), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_swiglu_quantize", rc)


def s3r_grouped_workspace(desc: QDesc, groups: int, d_in: int) -> int:
    return lib().s3r_grouped_workspace(ctypes.byref(desc), groups, d_in)


def _nbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def s3r_grouped_quantize(desc: QDesc, offsets, G, row_scale, col_scale, Q, delta, code_colsum=None, ec_row=None,
                         ec_col=None, ec_mean=None, flags=None, ws=None, stream=None, *, rc_only=False):
    """offsets: int64 device tensor [groups + 1]; col_scale [groups x D] (or None)."""
    rc = lib().s3r_grouped_quantize(ctypes.byref(desc), offsets.numel() - 1, _ptr(offsets), _ptr(G),
                                    _gdtype(G) if G is not None else S3R_F32, _ld(G, desc.cols), _ptr(row_scale),
                                    _ptr(col_scale), _ptr(Q), _ld(Q, desc.cols), _ptr(delta), _ptr(code_colsum),
                                    _ptr(ec_row), _ptr(ec_col), _ptr(ec_mean), _ptr(flags), _ptr(ws), _nbytes(ws),
                                    _stream(stream))
    if rc_only:
        return rc
    _check("s3r_grouped_quantize", rc)


def s3r_grouped_backward_dx(desc: QDesc, offsets, Q, delta, Wq, s_x, r_W, ec_row, ec_col, ec_mean, dX, flags=None,
                            ws=None, stream=None, *, accumulate=False, rc_only=False):
    """Wq: int8 [groups x D x d_in] (3-D, rows with unit stride)."""
    d_in = dX.shape[1]
    if Wq.dim() != 3 or Wq.stride(2) != 1:
        raise ValueError("expected Wq as [groups x D x d_in] with unit column stride")
    rc = lib().s3r_grouped_backward_dx(ctypes.byref(desc), offsets.numel() - 1, _ptr(offsets), _ptr(Q),
                                       _ld(Q, desc.cols), _ptr(delta), _ptr(Wq), Wq.stride(1), Wq.stride(0), d_in,
                                       _ptr(s_x), _ptr(r_W), _ptr(ec_row), _ptr(ec_col), _ptr(ec_mean), _ptr(dX),
                                       _odtype(dX, accumulate), _ld(dX, d_in), _ptr(flags), _ptr(ws), _nbytes(ws),
                                       _stream(stream))
    if rc_only:
        return rc
    _check("s3r_grouped_backward_dx", rc)


def s3r_grouped_backward_dw(desc: QDesc, offsets, Q, delta, Xq, s_w, xs, ec_row, ec_col, ec_mean, dW, flags=None,
                            ws=None, stream=None, *, rc_only=False):
    """dW: float32 / int32 [groups x D x d_in] (3-D, unit column stride)."""
    d_in = Xq.shape[1]
    if dW.dim() != 3 or dW.stride(2) != 1:
        raise ValueError("expected dW as [groups x D x d_in] with unit column stride")
    rc = lib().s3r_grouped_backward_dw(ctypes.byref(desc), offsets.numel() - 1, _ptr(offsets), _ptr(Q),
                                       _ld(Q, desc.cols), _ptr(delta), _ptr(Xq), _ld(Xq, d_in), d_in, _ptr(s_w),
                                       _ptr(xs), _ptr(ec_row), _ptr(ec_col), _ptr(ec_mean), _ptr(dW), _odtype(dW),
                                       dW.stride(1), dW.stride(0), _ptr(flags), _ptr(ws), _nbytes(ws),
                                       _stream(stream))
    if rc_only:
        return rc
    _check("s3r_grouped_backward_dw", rc)


def s3r_mx_workspace(desc: QDesc, d_in: int) -> int:
    return lib().s3r_mx_workspace(ctypes.byref(desc), d_in)


def s3r_mx_operand_workspace(rows: int, cols: int) -> int:
    return lib().s3r_mx_operand_workspace(rows, cols)


def s3r_mx_operand(M, Mt, Mt_scales, colsum=None, rows_per_example=None, flags=None, ws=None, stream=None, *,
                   rc_only=False):
    """M [rows x cols] f32/bf16 -> Mt (mx_codes(cols, rows)), Mt_scales uint8 [rows/128 x 4*cols] (step-grouped)."""
    rows, cols = M.shape
    S = rows if rows_per_example is None else rows_per_example
    rc = lib().s3r_mx_operand(rows, cols, S, _ptr(M), _gdtype(M), _ld(M, cols), _ptr(Mt), _ld(Mt),
                              _ptr(Mt_scales), _ld(Mt_scales, 4 * cols), _ptr(colsum), _ptr(flags), _ptr(ws),
                              _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_mx_operand", rc)


def s3r_mx_quantize(desc: QDesc, G, Qh, Qh_scales, Qt, Qt_scales, ec_row_h=None, ec_col_h=None, ec_mean_h=None,
                    ec_row_t=None, ec_col_t=None, ec_mean_t=None, flags=None, ws=None, stream=None, *,
                    rc_only=False):
    T, D = desc.rows, desc.cols
    rc = lib().s3r_mx_quantize(ctypes.byref(desc), _ptr(G), _gdtype(G) if G is not None else S3R_F32, _ld(G, D),
                               _ptr(Qh), _ld(Qh), _ptr(Qh_scales), _ld(Qh_scales, 4 * T), _ptr(Qt),
                               _ld(Qt), _ptr(Qt_scales), _ld(Qt_scales, 4 * D), _ptr(ec_row_h),
                               _ptr(ec_col_h), _ptr(ec_mean_h), _ptr(ec_row_t), _ptr(ec_col_t), _ptr(ec_mean_t),
                               _ptr(flags), _ptr(ws), _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_mx_quantize", rc)


def s3r_mx_backward_dx(desc: QDesc, Qh, Qh_scales, Wt, Wt_scales, r_W, ec_row_h, ec_col_h, ec_mean_h, dX, ws=None,
                       stream=None, *, rc_only=False):
    """Wt: mx_codes(d_in, D), Wt_scales [D/128 x 4*d_in]; dX f32 [T x d_in]."""
    d_in = dX.shape[1]
    rc = lib().s3r_mx_backward_dx(ctypes.byref(desc), _ptr(Qh), _ld(Qh), _ptr(Qh_scales),
                                  _ld(Qh_scales, 4 * desc.rows), _ptr(Wt), _ld(Wt), _ptr(Wt_scales),
                                  _ld(Wt_scales, 4 * d_in), d_in, _ptr(r_W), _ptr(ec_row_h), _ptr(ec_col_h),
                                  _ptr(ec_mean_h), _ptr(dX), _ld(dX, d_in), _ptr(ws), _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_mx_backward_dx", rc)


def s3r_mx_backward_dw(desc: QDesc, Qt, Qt_scales, Xt, Xt_scales, xs, ec_row_t, ec_col_t, ec_mean_t, dW, ws=None,
                       stream=None, *, rc_only=False):
    """Xt: mx_codes(d_in, T), Xt_scales [T/128 x 4*d_in]; dW f32 [D x d_in]."""
    d_in = dW.shape[1]
    rc = lib().s3r_mx_backward_dw(ctypes.byref(desc), _ptr(Qt), _ld(Qt), _ptr(Qt_scales),
                                  _ld(Qt_scales, 4 * desc.cols), _ptr(Xt), _ld(Xt), _ptr(Xt_scales),
                                  _ld(Xt_scales, 4 * d_in), d_in, _ptr(xs), _ptr(ec_row_t), _ptr(ec_col_t),
                                  _ptr(ec_mean_t), _ptr(dW), _ld(dW, d_in), _ptr(ws), _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_mx_backward_dw", rc)


def _typed(t, dtype, what):
    if t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")


def _shaped(t, shape, what):
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def s3r_route_workspace(desc: RouteDesc) -> int:
    return lib().s3r_route_workspace(ctypes.byref(desc))


def _flat(what, t, dtype, n):
    """Refuse t unless it is n contiguous elements of dtype."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous elements of {dtype}, got {t.dtype} {tuple(t.shape)}")


def s3r_route(desc: RouteDesc, logits, bias, ids, weights, offsets, slot_row, row_slot, ws, stream=None, *,
              rc_only=False):
    """logits [T x E] f32/bf16, bias f32 [E] or None -> ids int32 [T x k], weights f32 [T x k], offsets int64
    [E + 1], slot_row int32 [T x k], row_slot int32 [T * k]."""
    import torch
    T, E, k = desc.tokens, desc.experts, desc.top_k
    n, i32, f32 = T * k, torch.int32, torch.float32
    _shaped(logits, (T, E), "logits")
    if bias is not None:
        _flat("bias", bias, f32, E)
    _flat("ids", ids, i32, n)
    _flat("weights", weights, f32, n)
    _flat("offsets", offsets, torch.int64, E + 1)
    _flat("slot_row", slot_row, i32, n)
    _flat("row_slot", row_slot, i32, n)
    rc = lib().s3r_route(desc, logits.data_ptr(), _gdtype(logits), _ld(logits), _ptr(bias), ids.data_ptr(),
                         weights.data_ptr(), offsets.data_ptr(), slot_row.data_ptr(), row_slot.data_ptr(), _ptr(ws),
                         _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    if rc:
        _check("s3r_route", rc)


def s3r_route_backward(desc: RouteDesc, logits, ids, dweights, dlogits, stream=None, *, rc_only=False):
    """dlogits [T x E], of the logits' dtype, from dweights f32 [T x k] at the choice ids int32 [T x k]."""
    import torch
    T, E = shape = desc.tokens, desc.experts
    n = T * desc.top_k
    _shaped(logits, shape, "logits")
    _shaped(dlogits, shape, "dlogits")
    _typed(dlogits, logits.dtype, "dlogits")
    _flat("ids", ids, torch.int32, n)
    _flat("dweights", dweights, torch.float32, n)
    rc = lib().s3r_route_backward(desc, logits.data_ptr(), _gdtype(logits), _ld(logits), ids.data_ptr(),
                                  dweights.data_ptr(), dlogits.data_ptr(), _ld(dlogits), _stream(stream))
    if rc_only:
        return rc
    if rc:
        _check("s3r_route_backward", rc)


def _slots(slot_row, tokens):
    """(T, k) of a slot table that fits the token rows."""
    import torch
    shape = slot_row.shape
    if slot_row.dtype is not torch.int32 or len(shape) != 2 or shape[0] != tokens.shape[0] or \
            not slot_row.is_contiguous():
        raise ValueError("slot_row: expected a contiguous int32 [T x k]")
    return shape


def s3r_dispatch(X, slot_row, rows, stream=None, *, rc_only=False):
    """rows[slot_row[t, j]] = X[t]; rows [R x D] of X's dtype."""
    T, k = _slots(slot_row, X)
    _typed(rows, X.dtype, "rows")
    R, D = rows.shape
    if X.shape[1] != D:
        raise ValueError("X and rows differ in width")
    rc = lib().s3r_dispatch(T, k, R, D, _gdtype(X), X.data_ptr(), _ld(X), slot_row.data_ptr(), rows.data_ptr(), _ld(rows),
                            _stream(stream))
    if rc_only:
        return rc
    if rc:
        _check("s3r_dispatch", rc)


def s3r_combine(rows, slot_row, weights, y, stream=None, *, rc_only=False):
    """y[t] = sum_j weights[t, j] rows[slot_row[t, j]] (weights f32 [T x k], or None: 1)."""
    import torch
    T, k = _slots(slot_row, y)
    _typed(y, rows.dtype, "y")
    R, D = rows.shape
    if y.shape[1] != D:
        raise ValueError("rows and y differ in width")
    if weights is not None:
        _shaped(weights, (T, k), "weights")
        _flat("weights", weights, torch.float32, T * k)
    rc = lib().s3r_combine(T, k, R, D, _gdtype(rows), rows.data_ptr(), _ld(rows), slot_row.data_ptr(), _ptr(weights),
                           y.data_ptr(), _ld(y), _stream(stream))
    if rc_only:
        return rc
    if rc:
        _check("s3r_combine", rc)


def s3r_combine_backward(dy, rows, slot_row, weights, drows, dweights, stream=None, *, rc_only=False):
    """drows[slot_row[t, j]] = weights[t, j] dy[t]; dweights[t, j] = <dy[t], rows[slot_row[t, j]]>."""
    import torch
    T, k = shape = _slots(slot_row, dy)
    (R, D), dt, f32 = rows.shape, dy.dtype, torch.float32
    _typed(rows, dt, "rows")
    _typed(drows, dt, "drows")
    _shaped(drows, (R, D), "drows")
    if dy.shape[1] != D:
        raise ValueError("dy and rows differ in width")
    ld = _ld(rows)
    if _ld(drows) != ld:
        raise ValueError("rows and drows must share their layout")
    _shaped(weights, shape, "weights")
    _shaped(dweights, shape, "dweights")
    _flat("weights", weights, f32, T * k)
    _flat("dweights", dweights, f32, T * k)
    rc = lib().s3r_combine_backward(T, k, R, D, _gdtype(dy), dy.data_ptr(), _ld(dy), rows.data_ptr(), slot_row.data_ptr(),
                                    weights.data_ptr(), drows.data_ptr(), ld, dweights.data_ptr(), _stream(stream))
    if rc_only:
        return rc
    if rc:
        _check("s3r_combine_backward", rc)


@dataclass
class MxRows:
    """MXFP4 matrices of rows x K elements in the library's block layout, K padded to steps of 128:
    codes uint8 [groups x ceil(rows/256) x 16384 steps], scales uint8 [groups x steps x 4 rows]."""
    codes: object
    scales: object
    rows: int
    K: int
    groups: int = 1
    _descs: dict = field(default_factory=dict, repr=False)      # product descriptors by their sizes


def mx_rows_buffer(rows: int, K: int, device, groups: int = 1) -> MxRows:
    import torch
    steps = (K + 127) // 128
    u8 = dict(dtype=torch.uint8, device=device)
    return MxRows(torch.empty(groups, (rows + 255) // 256, 16384 * steps, **u8),
                  torch.empty(groups, steps, 4 * rows, **u8), rows, K, groups)


def _mx_fit(m: MxRows):
    """Refuse codes and scales that are smaller than m says (negative sizes are the library's to refuse)."""
    rows, codes, scales = m.rows, m.codes, m.scales
    n = m.groups * ((m.K + 127) // 128)
    if codes.nbytes < n * 16384 * ((rows + 255) // 256) or scales.nbytes < 4 * n * rows or \
            not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("MXFP4 codes or scales are not contiguous, or smaller than their rows")


def _index(index, rows):
    if index is not None:
        import torch
        _flat("index", index, torch.int32, rows)


def _like(A, up):
    if up is not None and (up.dtype != A.dtype or up.shape != A.shape or up.stride() != A.stride()):
        raise ValueError("up must have A's type, shape and layout")


def s3r_mx_rows(A, out: MxRows, up=None, index=None, index_div=1, flags=None, stream=None, *, rc_only=False):
    """A [rows x K], or [groups x rows x K], f32/bf16 (silu(A) * up with up) -> out; with index, row r of out is
    row index[r] // index_div of the 2-D A."""
    if A.dim() not in (2, 3) or A.stride(-1) != 1:
        raise ValueError("expected row-major matrices (unit column stride)")
    G, a_rows, K = (1, *A.shape) if A.dim() == 2 else A.shape
    if (out.groups, out.K) != (G, K) or (index is None and out.rows != a_rows):
        raise ValueError("out does not fit A")
    _mx_fit(out)
    _index(index, out.rows)
    _like(A, up)
    steps, blocks = (K + 127) // 128, (out.rows + 255) // 256
    rc = lib().s3r_mx_rows(G, out.rows, K, _ptr(A), _ptr(up), _gdtype(A), A.stride(-2), A.stride(0) if A.dim() == 3 else 0,
                           a_rows, _ptr(index), index_div, _ptr(out.codes), 16384 * steps, blocks * 16384 * steps,
                           _ptr(out.scales), 4 * out.rows, steps * 4 * out.rows, _ptr(flags), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_mx_rows", rc)


def _mx_pdesc(rows, w: MxRows, out, offsets):
    import torch
    dt = out.dtype
    _shaped(out, (rows, w.rows), "out")
    if offsets is None:
        if w.groups != 1:
            raise ValueError("several weights need the rows' offsets")
    else:
        _flat("offsets", offsets, torch.int64, w.groups + 1)
    key = rows, dt, offsets is None, w.rows, w.K, w.groups
    d = w._descs.get(key)
    if d is None:
        if dt not in (torch.float32, torch.bfloat16):
            raise ValueError(f"unsupported output dtype {dt}")
        steps, blocks = (w.K + 127) // 128, (w.rows + 255) // 256
        if len(w._descs) >= 64:         # a program with ever new row counts
            w._descs.clear()
        d = w._descs[key] = MxPDesc(rows, w.rows, w.K, 0 if offsets is None else w.groups, 16384 * steps, 4 * w.rows,
                                    blocks * 16384 * steps, steps * 4 * w.rows,
                                    S3R_BF16 if dt is torch.bfloat16 else S3R_F32, 0)
    return d


def s3r_mx_product(a: MxRows, w: MxRows, out, offsets=None, flags=None, stream=None, *, rc_only=False):
    """out [rows x w.rows] (f32/bf16) = a w^T; with offsets int64 [groups + 1], a's rows are sorted by group and
    group e takes w's matrix e."""
    if a.groups != 1 or a.K != w.K:
        raise ValueError("a and w do not fit")
    _mx_fit(a)
    _mx_fit(w)
    d = _mx_pdesc(a.rows, w, out, offsets)
    rc = lib().s3r_mx_product(d, _ptr(a.codes), 16384 * ((a.K + 127) // 128), _ptr(a.scales), 4 * a.rows,
                              _ptr(offsets), _ptr(w.codes), _ptr(w.scales), _ptr(out), _ld(out), _ptr(flags),
                              _stream(stream))
    if rc_only:
        return rc
    _check("s3r_mx_product", rc)


def s3r_mx_linear_workspace(rows: int, K: int) -> int:
    return lib().s3r_mx_linear_workspace(rows, K)


def mx_linear_buffer(rows: int, K: int, device):
    """A workspace for s3r_mx_linear on that many rows."""
    return _scratch(s3r_mx_linear_workspace(rows, K), device)


def s3r_mx_linear(A, w: MxRows, out, *, up=None, offsets=None, index=None, index_div=1, ws=None, flags=None,
                  stream=None, rc_only=False):
    """out = mx(A) w^T in one call (A as in s3r_mx_rows, the product as in s3r_mx_product)."""
    rows = out.shape[0]
    a_rows, K = A.shape
    if K != w.K or (index is None and a_rows != rows):
        raise ValueError("A, w and out do not fit")
    _mx_fit(w)
    _index(index, rows)
    _like(A, up)
    d = _mx_pdesc(rows, w, out, offsets)
    rc = lib().s3r_mx_linear(d, A.data_ptr(), _ptr(up), _gdtype(A), _ld(A), a_rows, _ptr(index), index_div, _ptr(offsets),
                             w.codes.data_ptr(), w.scales.data_ptr(), out.data_ptr(), _ld(out), _ptr(flags), _ptr(ws),
                             _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    if rc:
        _check("s3r_mx_linear", rc)


def _here(*tensors):
    """Refuse tensors of another device than the current one (the library works on that), or of the host."""
    import torch
    first = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != first:
            raise ValueError("tensors on different devices")
    if torch.cuda.is_available() if first < 0 else first != torch._C._cuda_getDevice():
        raise ValueError("tensors are not on the current device")


def _whole(t):
    """t, without elements contiguous (torch gives such tensors any strides)."""
    return t if t is None or t.numel() else t.new_empty(t.shape)


@dataclass
class IntRows:
    """INT8 matrices of rows x K codes, a step a row: codes int8 [groups x rows x K in whole 16s], delta f32
    [groups x rows].  ``Q`` is the codes as the backward's products take them."""
    codes: object
    delta: object
    rows: int
    K: int
    groups: int = 1
    _descs: dict = field(default_factory=dict, repr=False)      # product descriptors by their sizes

    @property
    def Q(self):
        q = self.codes[..., :self.K]
        return q[0] if self.groups == 1 else q


def int_rows_buffer(rows: int, K: int, device, groups: int = 1) -> IntRows:
    import torch
    return IntRows(torch.empty(groups, rows, _pad16(K), dtype=torch.int8, device=device),
                  torch.empty(groups, rows, dtype=torch.float32, device=device), rows, K, groups)


def _int_fit(m: IntRows):
    """Refuse codes and steps that are not what m says."""
    import torch
    c, d = m.codes, m.delta
    _typed(c, torch.int8, "codes")
    _typed(d, torch.float32, "delta")
    if c.shape != (m.groups, m.rows, _pad16(m.K)) or d.shape != (m.groups, m.rows) or not c.is_contiguous() or \
            not d.is_contiguous():
        raise ValueError("INT8 codes or steps are not contiguous, or not of their rows' sizes")


def s3r_int_rows(A, out: IntRows, up=None, index=None, index_div=1, flags=None, stream=None, *, rc_only=False):
    """A [rows x K], or [groups x rows x K], f32/bf16 (silu(A) * up with up) -> out; with index, row r of out is
    row index[r] // index_div of the 2-D A."""
    A, up = _whole(A), _whole(up)
    if A.dim() not in (2, 3) or A.stride(-1) != 1:
        raise ValueError("expected row-major matrices (unit column stride)")
    G, a_rows, K = (1, *A.shape) if A.dim() == 2 else A.shape
    if (out.groups, out.K) != (G, K) or (index is None and out.rows != a_rows):
        raise ValueError("out does not fit A")
    _int_fit(out)
    _index(index, out.rows)
    _like(A, up)
    _here(A, out.codes, out.delta, up, index, flags)
    ld = _pad16(K)
    rc = lib().s3r_int_rows(G, out.rows, K, _ptr(A), _ptr(up), _gdtype(A), A.stride(-2), A.stride(0) if A.dim() == 3 else 0,
                           a_rows, _ptr(index), index_div, _ptr(out.codes), ld, out.rows * ld, _ptr(out.delta), _ptr(flags),
                           _stream(stream))
    if rc_only:
        return rc
    _check("s3r_int_rows", rc)


def s3r_int_colsum(Q, sums, offsets=None, flags=None, stream=None, *, rc_only=False):
    """sums int32 [groups x K] of the codes Q [rows x K] over each group's rows (offsets int64 [groups + 1]), or over
    equal runs of rows."""
    import torch
    _typed(Q, torch.int8, "Q")
    rows, K = Q.shape
    groups = sums.shape[0]
    _typed(sums, torch.int32, "sums")
    _shaped(sums, (groups, K), "sums")
    if not sums.is_contiguous():
        raise ValueError("sums: expected a contiguous tensor")
    if offsets is not None:
        _flat("offsets", offsets, torch.int64, groups + 1)
    _here(Q, sums, offsets, flags)
    rc = lib().s3r_int_colsum(groups, _ptr(offsets), rows, K, _ptr(Q), _ld(Q), _ptr(sums), _ptr(flags), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_int_colsum", rc)


def _int_pdesc(rows, w: IntRows, out, offsets, bias):
    import torch
    dt = out.dtype
    _shaped(out, (rows, w.rows), "out")
    if offsets is None:
        if w.groups != 1:
            raise ValueError("several weights need the rows' offsets")
    else:
        _flat("offsets", offsets, torch.int64, w.groups + 1)
    if bias is not None:
        _flat("bias", bias, torch.float32, w.groups * w.rows)
    key = rows, dt, offsets is None, w.rows, w.K, w.groups
    d = w._descs.get(key)
    if d is None:
        if dt not in (torch.float32, torch.bfloat16):
            raise ValueError(f"unsupported output dtype {dt}")
        if len(w._descs) >= 64:         # a program with ever new row counts
            w._descs.clear()
        ld = _pad16(w.K)
        d = w._descs[key] = IntPDesc(rows, w.rows, w.K, 0 if offsets is None else w.groups, ld, w.rows * ld,
                                    S3R_BF16 if dt is torch.bfloat16 else S3R_F32, 0)
    return d


def s3r_int_product(a: IntRows, w: IntRows, out, offsets=None, bias=None, flags=None, stream=None, *, rc_only=False):
    """out [rows x w.rows] (f32/bf16) = a w^T + bias; with offsets int64 [groups + 1], a's rows are sorted by group and
    group e takes w's matrix e and bias[e] (f32 [w.rows], or [groups x w.rows])."""
    if a.groups != 1 or a.K != w.K:
        raise ValueError("a and w do not fit")
    _int_fit(a)
    _int_fit(w)
    _here(a.codes, a.delta, w.codes, w.delta, out, offsets, bias, flags)
    d = _int_pdesc(a.rows, w, out, offsets, bias)
    rc = lib().s3r_int_product(d, _ptr(a.codes), _pad16(a.K), _ptr(a.delta), _ptr(offsets), _ptr(w.codes), _ptr(w.delta),
                              _ptr(bias), _ptr(out), _ld(out), _ptr(flags), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_int_product", rc)


def s3r_int_linear_workspace(rows: int, K: int) -> int:
    return lib().s3r_int_linear_workspace(rows, K)


def int_linear_buffer(rows: int, K: int, device):
    """A workspace for s3r_int_linear on that many rows."""
    return _scratch(s3r_int_linear_workspace(rows, K), device)


def s3r_int_linear(A, w: IntRows, out, *, up=None, offsets=None, index=None, index_div=1, bias=None, ws=None, flags=None,
                  stream=None, rc_only=False):
    """out = int8(A) w^T + bias in one call (A as in s3r_int_rows, the product as in s3r_int_product)."""
    rows = out.shape[0]
    A, up = _whole(A), _whole(up)
    a_rows, K = A.shape
    if K != w.K or (index is None and a_rows != rows):
        raise ValueError("A, w and out do not fit")
    _int_fit(w)
    _index(index, rows)
    _like(A, up)
    _here(A, w.codes, w.delta, out, up, offsets, index, bias, ws, flags)
    d = _int_pdesc(rows, w, out, offsets, bias)
    rc = lib().s3r_int_linear(d, A.data_ptr(), _ptr(up), _gdtype(A), _ld(A), a_rows, _ptr(index), index_div, _ptr(offsets),
                             w.codes.data_ptr(), w.delta.data_ptr(), _ptr(bias), out.data_ptr(), _ld(out), _ptr(flags),
                             _ptr(ws), _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    if rc:
        _check("s3r_int_linear", rc)


NS_COEFFS = (3.4445, -4.7750, 2.0315)


def orth_desc(shape, g_dtype=S3R_F32, out_dtype=S3R_F32, *, steps=5, coeffs=NS_COEFFS, eps=1e-7, scale=1.0,
              keep=0.0) -> OrthDesc:
    """Of matrices [rows x cols] or [groups x rows x cols]."""
    groups, rows, cols = (1, *shape) if len(shape) == 2 else shape
    a, b, c = coeffs
    return OrthDesc(groups, rows, cols, g_dtype, out_dtype, steps, a, b, c, eps, scale, keep, 0)


def s3r_orthogonalize_workspace(desc: OrthDesc) -> int:
    return lib().s3r_orthogonalize_workspace(desc)


def orthogonalize_buffer(G):
    """A workspace for s3r_orthogonalize on matrices of G's shape."""
    return _scratch(s3r_orthogonalize_workspace(orth_desc(G.shape)), G.device)


def s3r_orthogonalize(G, out, *, steps=5, coeffs=NS_COEFFS, eps=1e-7, scale=1.0, keep=0.0, ws=None, stream=None,
                      rc_only=False):
    """out = keep out + scale X, X the Newton-Schulz steps' result of G [rows x cols] or [groups x rows x cols] (f32/bf16,
    out too); out may be G."""
    G, out = _whole(G), _whole(out)
    if G.dim() not in (2, 3):
        raise ValueError("expected a matrix, or several")
    _shaped(out, G.shape, "out")
    if G.stride(-1) != 1 or out.stride(-1) != 1:
        raise ValueError("expected row-major matrices (unit column stride)")
    _here(G, out, ws)
    d = orth_desc(G.shape, _gdtype(G), _gdtype(out), steps=steps, coeffs=coeffs, eps=eps, scale=scale, keep=keep)
    many = G.dim() == 3
    rc = lib().s3r_orthogonalize(d, _ptr(G), G.stride(-2), G.stride(0) if many else 0, _ptr(out), out.stride(-2),
                                 out.stride(0) if many else 0, _ptr(ws), _nbytes(ws), _stream(stream))
    if rc_only:
        return rc
    _check("s3r_orthogonalize", rc)


def swiglu_backward(dH, A_gate, A_up, stream=None):
    """Allocate G_gate, G_up (bf16, like A_gate) and run s3r_swiglu_backward."""
    import torch
    G_gate = torch.empty(A_gate.shape, dtype=torch.bfloat16, device=A_gate.device)
    G_up = torch.empty_like(G_gate)
    s3r_swiglu_backward(dH, A_gate, A_up, G_gate, G_up, stream)
    return G_gate, G_up


def swiglu_quantize(dH, A_gate, A_up, *, mode=S3R, ec=EC_NONE, row_scale=None, col_scale_gate=None,
                    col_scale_up=None, seed=0, layer_gate=0, layer_up=0, rows_per_example=None, stream=None,
                    threshold_stream=0):
    """Allocate the outputs and run s3r_swiglu_quantize: (Quantized gate, Quantized up)."""
    import torch
    T, F = dH.shape
    dev = dH.device
    dg = qdesc(T, F, rows_per_example, mode, ec, PER_TENSOR, layer_gate, seed, threshold_stream)
    du = qdesc(T, F, rows_per_example, mode, ec, PER_TENSOR, layer_up, seed, threshold_stream)
    B = T // dg.rows_per_example
    out = []
    for d in (dg, du):
        e = (None, None, None)
        if ec != EC_NONE:
            e = (torch.empty(T, dtype=torch.float32, device=dev), torch.empty(B, F, dtype=torch.float32, device=dev),
                 torch.empty(B, dtype=torch.float32, device=dev))
        out.append((q_buffer(T, F, dev), torch.empty(1, dtype=torch.float32, device=dev), e))
    flags = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = _workspace(s3r_swiglu_quantize_workspace(dg), dev)
    s3r_swiglu_quantize(dg, du, dH, A_gate, A_up, row_scale, col_scale_gate, col_scale_up, out[0][0], out[1][0],
                        out[0][1], out[1][1], out[0][2], out[1][2], flags, ws, stream)
    return (Quantized(out[0][0], out[0][1], dg, None, *out[0][2], flags),
            Quantized(out[1][0], out[1][1], du, None, *out[1][2], flags))


def s3r_time_next_gemm(start_event, stop_event) -> None:
    """Record two torch.cuda.Event objects around the next GEMM kernel launched from this thread."""
    _check("s3r_time_next_gemm", lib().s3r_time_next_gemm(
        ctypes.c_void_p(start_event.cuda_event) if start_event is not None else None,
        ctypes.c_void_p(stop_event.cuda_event) if stop_event is not None else None))


def s3r_version() -> int:
    return lib().s3r_version()


def s3r_status_string(code: int) -> str:
    return lib().s3r_status_string(code).decode()


# ------------------------------------------------------ allocating helpers ----

def _pad16(n: int) -> int:
    return (n + 15) // 16 * 16


def _workspace(nbytes: int, device):
    import torch
    return torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=device) if nbytes else None


def q_buffer(rows: int, cols: int, device):
    """int8 [rows x cols] view with a leading dimension padded to 16 (what the GEMMs need)."""
    import torch
    return torch.empty(rows, _pad16(cols), dtype=torch.int8, device=device)[:, :cols]


@dataclass
class Quantized:
    Q: object            # int8 [T x D] (leading dim padded to 16)
    delta: object        # f32 [1] or [T]
    desc: QDesc
    code_colsum: object = None
    ec_row: object = None
    ec_col: object = None
    ec_mean: object = None
    flags: object = None


def quantize(G, *, mode=S3R, ec=EC_NONE, scale=PER_TENSOR, row_scale=None, col_scale=None, seed=0, layer_id=0,
             rows_per_example=None, colsum=False, stream=None, threshold_stream=0) -> Quantized:
    import torch
    T, D = G.shape
    desc = qdesc(T, D, rows_per_example, mode, ec, scale, layer_id, seed, threshold_stream)
    dev = G.device
    S = desc.rows_per_example
    B = T // S
    Q = q_buffer(T, D, dev)
    delta = torch.empty(T if scale == PER_TOKEN else 1, dtype=torch.float32, device=dev)
    cs = torch.empty(B, D, dtype=torch.int32, device=dev) if colsum else None
    e_r = e_c = e_m = None
    if ec != EC_NONE:
        e_r = torch.empty(T, dtype=torch.float32, device=dev)
        e_c = torch.empty(B, D, dtype=torch.float32, device=dev)
        e_m = torch.empty(B, dtype=torch.float32, device=dev)
    flags = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = _workspace(s3r_quantize_workspace(desc), dev)
    s3r_quantize(desc, G, row_scale, col_scale, Q, delta, cs, e_r, e_c, e_m, flags, ws, stream)
    return Quantized(Q, delta, desc, cs, e_r, e_c, e_m, flags)


def forward_operand(X, rows_per_example=None, stream=None) -> Quantized:
    """Per-row absmax RTNE of a forward operand (X per token, W per output channel) with code column sums."""
    return quantize(X, mode=RTNE, ec=EC_NONE, scale=PER_TOKEN, rows_per_example=rows_per_example, colsum=True,
                    stream=stream)


def backward_dx(q: Quantized, Wq, s_x=None, r_W=None, out_dtype=None, stream=None, out=None):
    """dX of one projection; with ``out`` (f32) the result is added into it."""
    import torch
    d_in = Wq.shape[1]
    T = q.desc.rows
    dX = out if out is not None else torch.empty(T, d_in, dtype=out_dtype or torch.float32, device=Wq.device)
    ws = _workspace(s3r_backward_workspace(q.desc, d_in), Wq.device)
    s3r_backward_dx(q.desc, q.Q, q.delta, Wq, s_x, r_W, q.ec_row, q.ec_col, q.ec_mean, dX, ws, stream,
                    accumulate=out is not None)
    return dX


def backward_dw(q: Quantized, Xq, s_w=None, xs_b=None, out_dtype=None, stream=None):
    import torch
    d_in = Xq.shape[1]
    D = q.desc.cols
    dW = torch.empty(D, d_in, dtype=out_dtype or torch.float32, device=Xq.device)
    ws = _workspace(s3r_backward_workspace(q.desc, d_in), Xq.device)
    s3r_backward_dw(q.desc, q.Q, q.delta, Xq, s_w, xs_b, q.ec_row, q.ec_col, q.ec_mean, dW, ws, stream)
    return dW


def backward_dw_pair(qa: Quantized, qb: Quantized, Xq, s_w_a=None, s_w_b=None, xs_b=None, out_dtype=None,
                     stream=None):
    """dW of two projections of the input Xq (one GEMM launch); qa and qb share shape and layout."""
    import torch
    d_in = Xq.shape[1]
    D = qa.desc.cols
    dWa = torch.empty(D, d_in, dtype=out_dtype or torch.float32, device=Xq.device)
    dWb = torch.empty_like(dWa)
    ws = _workspace(s3r_backward_dw_pair_workspace(qa.desc, d_in), Xq.device)
    s3r_backward_dw_pair(qa.desc, qa.Q, qb.Q, qa.delta, qb.delta, Xq, s_w_a, s_w_b, xs_b,
                         (qa.ec_row, qa.ec_col, qa.ec_mean), (qb.ec_row, qb.ec_col, qb.ec_mean), dWa, dWb, ws, stream)
    return dWa, dWb


# ------------------------------------------------------------ MXFP4 helpers ----

def mx_codes(rows: int, K: int, device):
    """uint8 buffer for the MXFP4 codes of a rows x K matrix in the library's block layout:
    [ceil(rows/256) x 128*K], one row per 256-row block (its stride is the layout's ld)."""
    import torch
    return torch.empty((rows + 255) // 256, 128 * K, dtype=torch.uint8, device=device)


@dataclass
class MxQuantized:
    Qh: object           # mx_codes(T, D): E2M1 codes, blocks along D
    Qh_scales: object    # uint8 [D/128 x 4T] E8M0, step-grouped
    Qt: object           # mx_codes(D, T): codes of G^T, blocks along T
    Qt_scales: object    # uint8 [T/128 x 4D]
    desc: QDesc
    ec_h: tuple = (None, None, None)   # (eps_t [T], ebar [B x D], mu [B]) of Q_h's error
    ec_t: tuple = (None, None, None)   # the same for Q_t
    flags: object = None


def mx_quantize(G, *, mode=S3R, ec=EC_NONE, seed=0, layer_id=0, rows_per_example=None, stream=None,
                threshold_stream=0) -> MxQuantized:
    import torch
    T, D = G.shape
    desc = qdesc(T, D, rows_per_example, mode, ec, PER_TENSOR, layer_id, seed, threshold_stream)
    dev = G.device
    B = T // desc.rows_per_example
    u8 = dict(dtype=torch.uint8, device=dev)
    Qh, Qhs = mx_codes(T, D, G.device), torch.empty(D // 128, 4 * T, **u8)
    Qt, Qts = mx_codes(D, T, G.device), torch.empty(T // 128, 4 * D, **u8)
    ec_h = ec_t = (None, None, None)
    if ec != EC_NONE:
        f32 = dict(dtype=torch.float32, device=dev)
        ec_h = (torch.empty(T, **f32), torch.empty(B, D, **f32), torch.empty(B, **f32))
        ec_t = (torch.empty(T, **f32), torch.empty(B, D, **f32), torch.empty(B, **f32))
    flags = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = _workspace(s3r_mx_workspace(desc, 0), dev)
    s3r_mx_quantize(desc, G, Qh, Qhs, Qt, Qts, *ec_h, *ec_t, flags, ws, stream)
    return MxQuantized(Qh, Qhs, Qt, Qts, desc, ec_h, ec_t, flags)


def mx_operand(M, rows_per_example=None, colsum=True, stream=None):
    """RTNE MXFP4 of a forward operand, stored transposed: (Mt, Mt_scales, colsum or None)."""
    import torch
    rows, cols = M.shape
    S = rows if rows_per_example is None else rows_per_example
    dev = M.device
    Mt = mx_codes(cols, rows, dev)
    Mts = torch.empty(rows // 128, 4 * cols, dtype=torch.uint8, device=dev)
    cs = torch.empty(rows // S, cols, dtype=torch.float32, device=dev) if colsum else None
    ws = _workspace(s3r_mx_operand_workspace(rows, cols), dev)
    s3r_mx_operand(M, Mt, Mts, cs, S, None, ws, stream)
    return Mt, Mts, cs


def mx_backward_dx(q: MxQuantized, Wt, Wt_scales, r_W=None, stream=None):
    import torch
    d_in = Wt_scales.shape[1] // 4
    dX = torch.empty(q.desc.rows, d_in, dtype=torch.float32, device=Wt.device)
    ws = _workspace(s3r_mx_workspace(q.desc, d_in), Wt.device)
    s3r_mx_backward_dx(q.desc, q.Qh, q.Qh_scales, Wt, Wt_scales, r_W, *q.ec_h, dX, ws, stream)
    return dX


def mx_backward_dw(q: MxQuantized, Xt, Xt_scales, xs=None, stream=None):
    import torch
    d_in = Xt_scales.shape[1] // 4
    dW = torch.empty(q.desc.cols, d_in, dtype=torch.float32, device=Xt.device)
    ws = _workspace(s3r_mx_workspace(q.desc, d_in), Xt.device)
    s3r_mx_backward_dw(q.desc, q.Qt, q.Qt_scales, Xt, Xt_scales, xs, *q.ec_t, dW, ws, stream)
    return dW


# ------------------------------------------- routing and expert-row helpers ----
# With ``stream`` (a raw handle) these allocate on that stream, so that neither their outputs nor a workspace that
# is freed on return can be handed to work of another stream too early; the inputs have to be ready there.

def _on(stream):
    if stream is None:
        return contextlib.nullcontext()
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream))


def _scratch(nbytes: int, device):
    import torch
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


@dataclass
class Routed:
    """A router's answer: the choice, its weights and the expert-sorted order of the rows."""
    ids: object          # int32 [T x k]
    weights: object      # f32 [T x k]
    offsets: object      # int64 [E + 1]: expert e owns rows offsets[e] .. offsets[e + 1]
    slot_row: object     # int32 [T x k]: the row of each slot
    row_slot: object     # int32 [T * k]: the slot of each row
    desc: RouteDesc = None
    ws: object = None


def routed_buffers(desc: RouteDesc, device) -> Routed:
    """Outputs and workspace for s3r_route, to be kept between calls."""
    import torch
    T, E, k = desc.tokens, desc.experts, desc.top_k
    i32 = dict(dtype=torch.int32, device=device)
    return Routed(torch.empty(T, k, **i32), torch.empty(T, k, dtype=torch.float32, device=device),
                  torch.empty(E + 1, dtype=torch.int64, device=device), torch.empty(T, k, **i32),
                  torch.empty(T * k, **i32), desc, _scratch(s3r_route_workspace(desc), device))


def route(logits, top_k, *, score=SOFTMAX, bias=None, groups=1, keep=1, group_top=1, renorm=True, scale=1.0,
          stream=None) -> Routed:
    """Choose top_k experts for every row of the logits [T x E]."""
    d = route_desc(*logits.shape, top_k, score=score, groups=groups, keep=keep, group_top=group_top, renorm=renorm,
                   scale=scale)
    with _on(stream):
        r = routed_buffers(d, logits.device)
    s3r_route(d, logits, bias, r.ids, r.weights, r.offsets, r.slot_row, r.row_slot, r.ws, stream)
    return r


def route_backward(r: Routed, logits, dweights, stream=None):
    """The logits' gradient from the weights'."""
    import torch
    with _on(stream):
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    s3r_route_backward(r.desc, logits, r.ids, dweights, dlogits, stream)
    return dlogits


def dispatch(X, r: Routed, stream=None):
    """The tokens' rows in the experts' order: [T * k x D].  Where r's slot_row was changed to leave rows out, they are
    not written (use s3r_dispatch on a cleared buffer)."""
    import torch
    with _on(stream):
        rows = torch.empty(r.row_slot.numel(), X.shape[1], dtype=X.dtype, device=X.device)
    s3r_dispatch(X, r.slot_row, rows, stream)
    return rows


def combine(rows, r: Routed, weighted=True, stream=None):
    """The experts' rows summed back into the tokens, weighted (or not: dispatch's gradient)."""
    import torch
    with _on(stream):
        y = torch.empty(r.ids.shape[0], rows.shape[1], dtype=rows.dtype, device=rows.device)
    s3r_combine(rows, r.slot_row, r.weights if weighted else None, y, stream)
    return y


def combine_backward(dy, rows, r: Routed, stream=None):
    """(drows, dweights) of combine(rows, r).  Rows past r's slots have the gradient 0; where r's slot_row was changed
    to leave rows out, theirs is not written (use s3r_combine_backward on a cleared buffer)."""
    import torch
    with _on(stream):
        drows = torch.empty_strided(rows.shape, rows.stride(), dtype=rows.dtype, device=rows.device)
        if rows.shape[0] > r.slot_row.numel():
            drows[r.slot_row.numel():].zero_()
        dw = torch.empty_like(r.weights)
    s3r_combine_backward(dy, rows, r.slot_row, r.weights, drows, dw, stream)
    return drows, dw


def mx_rows(A, *, up=None, index=None, index_div=1, flags=None, stream=None) -> MxRows:
    """RTNE MXFP4 of the rows of A ([rows x K], or [groups x rows x K]: weights [N x K] of every expert)."""
    G = 1 if A.dim() == 2 else A.shape[0]
    with _on(stream):
        out = mx_rows_buffer(A.shape[-2] if index is None else index.numel(), A.shape[-1], A.device, G)
    s3r_mx_rows(A, out, up, index, index_div, flags, stream)
    return out


def mx_product(a: MxRows, w: MxRows, *, offsets=None, out_dtype=None, flags=None, stream=None):
    import torch
    with _on(stream):
        out = torch.empty(a.rows, w.rows, dtype=out_dtype or torch.float32, device=a.codes.device)
    s3r_mx_product(a, w, out, offsets, flags, stream)
    return out


def mx_linear(A, w: MxRows, *, up=None, offsets=None, index=None, index_div=1, out_dtype=None, flags=None, stream=None):
    """A's rows in MXFP4 times the weights w (mx_rows): [rows x w.rows], of A's dtype unless out_dtype is given."""
    import torch
    rows = A.shape[0] if index is None else index.numel()
    with _on(stream):
        out = torch.empty(rows, w.rows, dtype=out_dtype or A.dtype, device=A.device)
        ws = mx_linear_buffer(rows, w.K, A.device)
    s3r_mx_linear(A, w, out, up=up, offsets=offsets, index=index, index_div=index_div, ws=ws, flags=flags, stream=stream)
    return out


# ------------------------------------------------- INT8 forward helpers ----
# ``stream`` as in the helpers above.

def int_rows(A, *, up=None, index=None, index_div=1, flags=None, stream=None) -> IntRows:
    """INT8 rows of A ([rows x K], or [groups x rows x K]: weights [N x K] of every expert), a step each (RTNE)."""
    G = 1 if A.dim() == 2 else A.shape[0]
    with _on(stream):
        out = int_rows_buffer(A.shape[-2] if index is None else index.numel(), A.shape[-1], A.device, G)
    s3r_int_rows(A, out, up, index, index_div, flags, stream)
    return out


def int_colsum(Q, groups=1, *, offsets=None, flags=None, stream=None):
    """Column sums of the codes Q [rows x K] over equal runs of rows, or over the groups of offsets: int32 [groups x K]."""
    import torch
    with _on(stream):
        sums = torch.empty(groups if offsets is None else offsets.numel() - 1, Q.shape[1], dtype=torch.int32, device=Q.device)
    s3r_int_colsum(Q, sums, offsets, flags, stream)
    return sums


def int_product(a: IntRows, w: IntRows, *, offsets=None, bias=None, out_dtype=None, flags=None, stream=None):
    import torch
    with _on(stream):
        out = torch.empty(a.rows, w.rows, dtype=out_dtype or torch.float32, device=a.codes.device)
    s3r_int_product(a, w, out, offsets, bias, flags, stream)
    return out


def int_linear(A, w: IntRows, *, up=None, offsets=None, index=None, index_div=1, bias=None, out_dtype=None, flags=None,
              stream=None):
    """A's rows in INT8 times the weights w (int_rows): [rows x w.rows], of A's dtype unless out_dtype is given."""
    import torch
    rows = A.shape[0] if index is None else index.numel()
    with _on(stream):
        out = torch.empty(rows, w.rows, dtype=out_dtype or A.dtype, device=A.device)
        ws = int_linear_buffer(rows, w.K, A.device)
    s3r_int_linear(A, w, out, up=up, offsets=offsets, index=index, index_div=index_div, bias=bias, ws=ws, flags=flags,
                  stream=stream)
    return out


def orthogonalize(G, *, steps=5, coeffs=NS_COEFFS, eps=1e-7, scale=1.0, out_dtype=None, stream=None):
    """G's singular values driven to about 1 by Newton-Schulz steps, times scale; of G's dtype unless out_dtype is given."""
    import torch
    with _on(stream):
        out = torch.empty(G.shape, dtype=out_dtype or G.dtype, device=G.device)
        ws = orthogonalize_buffer(G)
    s3r_orthogonalize(G, out, steps=steps, coeffs=coeffs, eps=eps, scale=scale, ws=ws, stream=stream)
    return out
