"""MI355X (gfx950) 2-D convolution forward: thin Python binding of libconvfwd.so.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/conv.h.  The names mirror the C
calls (conv_output_extent, conv_resolve_auto_pad, conv_scratch_size,
conv_describe_variant, conv_forward, conv_transpose_forward; the linear, gated
and grad_clip calls of include/linear.h and include/grad_clip.h).  Loading fails
loudly when the native library has not been built; there is no fallback.

Operands are device pointers (ints) or objects with a ``data_ptr()`` method
(torch tensors on the GPU).  PyTorch is only used by callers for device memory
and streams.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libconvfwd.so")

# enums of include/conv.h
CONV_OK, CONV_ERR_ARG, CONV_ERR_SHAPE, CONV_ERR_OVERLAP, CONV_ERR_SCRATCH, CONV_ERR_DEVICE = range(6)
CONV_F32, CONV_F16, CONV_BF16 = 0, 1, 2
DTYPES = {"f32": CONV_F32, "f16": CONV_F16, "bf16": CONV_BF16}
ACTIVATIONS = {
    "identity": 0, "relu": 1, "tanh": 2, "sigmoid": 3, "silu": 4,
    "hard_sigmoid": 5, "hard_swish": 6, "clip": 7, "leaky_relu": 8,
}
AUTO_PAD = {"NOTSET": 0, "SAME_UPPER": 1, "SAME_LOWER": 2, "VALID": 3}
VARIANTS = {
    "auto": 0, "implicit_gemm": 1, "pointwise_gemm": 2, "depthwise_direct": 3,
    "transpose_gemm_col2im": 4, "implicit_gemm_halo": 5, "implicit_gemm_rowband": 6,
    "implicit_gemm_grouped": 7, "winograd": 8,
}
# default activation parameters (ONNX): hard_sigmoid alpha/beta, leaky alpha
ACT_DEFAULTS = {"hard_sigmoid": (0.2, 0.5), "leaky_relu": (0.01, 0.0)}

EXPORTS = (
    "conv_output_extent", "conv_resolve_auto_pad", "conv_scratch_size",
    "conv_describe_variant", "conv_forward", "conv_transpose_forward",
    "conv_check", "conv_status_string", "conv_forward_noalloc",
    "pool_output_extent", "pool_resolve_auto_pad", "pool_describe_variant", "pool_check",
    "pool_forward", "conv_integer_describe_variant", "conv_integer_check", "conv_integer_forward",
    "linear_scratch_size", "linear_backward_scratch_size", "linear_describe_variant",
    "linear_backward_describe_variant", "linear_check", "linear_backward_check", "linear_forward",
    "linear_backward", "gated_scratch_size", "gated_backward_scratch_size",
    "gated_describe_variant", "gated_backward_describe_variant", "gated_check",
    "gated_backward_check", "gated_forward", "gated_backward",
    "grad_clip_scratch_size", "grad_clip_check", "grad_clip",
)


class ConvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


class conv_problem(ctypes.Structure):
    """Mirror of struct conv_problem in include/conv.h (same field order)."""

    _fields_ = [(n, ctypes.c_int64) for n in (
        "n", "c_in", "h", "w", "c_out", "kh", "kw", "groups",
        "stride_h", "stride_w", "dil_h", "dil_w",
        "pad_top", "pad_left", "pad_bottom", "pad_right",
        "out_pad_h", "out_pad_w",
        "x_off", "w_off", "b_off", "r_off", "y_off")] + [
        ("transpose", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("act_alpha", ctypes.c_float), ("act_beta", ctypes.c_float),
        ("has_bias", ctypes.c_int32), ("has_residual", ctypes.c_int32),
        ("variant_override", ctypes.c_int32), ("split_override", ctypes.c_int32)]


class pool_problem(ctypes.Structure):
    """Mirror of struct pool_problem in include/pool.h (same field order)."""

    _fields_ = [(n, ctypes.c_int64) for n in (
        "n", "c", "h", "w", "kh", "kw", "stride_h", "stride_w", "dil_h", "dil_w",
        "pad_top", "pad_left", "pad_bottom", "pad_right", "x_off", "y_off")] + [
        ("kind", ctypes.c_int32), ("ceil_mode", ctypes.c_int32),
        ("count_include_pad", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class linear_problem(ctypes.Structure):
    """Mirror of struct linear_problem in include/linear.h (same field order)."""

    _fields_ = [(n, ctypes.c_int64) for n in (
        "m", "n", "k", "ldx", "ldw", "ldr", "ldy", "ldz", "lddx", "lddw", "lddr",
        "x_off", "w_off", "b_off", "r_off", "y_off", "z_off",
        "dy_off", "dx_off", "dw_off", "db_off", "dr_off")] + [
        ("activation", ctypes.c_int32), ("act_alpha", ctypes.c_float),
        ("act_beta", ctypes.c_float), ("has_bias", ctypes.c_int32),
        ("has_residual", ctypes.c_int32), ("save_z", ctypes.c_int32),
        ("w_layout", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class gated_problem(ctypes.Structure):
    """Mirror of struct gated_problem in include/linear.h (same field order)."""

    _fields_ = [(n, ctypes.c_int64) for n in (
        "m", "f", "k", "ldx", "ldw", "ldh", "ldp", "lddx", "lddw",
        "x_off", "wg_off", "wu_off", "bg_off", "bu_off", "h_off", "pg_off", "pu_off",
        "dh_off", "dx_off", "dwg_off", "dwu_off", "dbg_off", "dbu_off")] + [
        ("activation", ctypes.c_int32), ("act_alpha", ctypes.c_float),
        ("act_beta", ctypes.c_float), ("has_bias", ctypes.c_int32),
        ("save_p", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class grad_tensor(ctypes.Structure):
    """Mirror of struct grad_tensor in include/grad_clip.h (same field order)."""

    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("elems", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class grad_clip_problem(ctypes.Structure):
    """Mirror of struct grad_clip_problem in include/grad_clip.h (same field order)."""

    _fields_ = [("tensors", ctypes.POINTER(grad_tensor)), ("count", ctypes.c_int64),
                ("kind", ctypes.c_int32), ("max_norm", ctypes.c_float), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


POOL_KINDS = {"max": 0, "average": 1, "global_max": 2, "global_average": 3}

_lib = None


def lib():
    """The loaded native library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with convolution_forward_amd.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(conv_problem)
        i64p = ctypes.POINTER(ctypes.c_int64)
        u64p = ctypes.POINTER(ctypes.c_uint64)
        vp = ctypes.c_void_p
        L.conv_output_extent.argtypes = [P, i64p, i64p]
        L.conv_resolve_auto_pad.argtypes = [P, ctypes.c_int, i64p]
        L.conv_scratch_size.argtypes = [P, ctypes.c_int, u64p, u64p]
        L.conv_describe_variant.argtypes = [P, ctypes.c_int, ctypes.c_char_p, ctypes.c_uint64]
        fwd = [P, ctypes.c_int, vp, vp, vp, vp, vp, vp, ctypes.c_uint64, vp]
        L.conv_forward.argtypes = fwd
        L.conv_transpose_forward.argtypes = fwd
        L.conv_check.argtypes = [P, ctypes.c_int, vp, vp, vp, vp, vp, vp, ctypes.c_uint64]
        L.conv_forward_noalloc.argtypes = [P, ctypes.c_int, vp, vp, vp, vp, vp, vp]
        PP = ctypes.POINTER(pool_problem)
        L.pool_output_extent.argtypes = [PP, i64p, i64p]
        L.pool_resolve_auto_pad.argtypes = [PP, ctypes.c_int]
        L.pool_describe_variant.argtypes = [PP, ctypes.c_int, ctypes.c_char_p, ctypes.c_uint64]
        L.pool_check.argtypes = [PP, ctypes.c_int, vp, vp]
        L.pool_forward.argtypes = [PP, ctypes.c_int, vp, vp, vp]
        L.conv_integer_describe_variant.argtypes = [P, ctypes.c_int, ctypes.c_int, ctypes.c_char_p,
                                                    ctypes.c_uint64]
        L.conv_integer_check.argtypes = [P, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp,
                                         ctypes.c_int, vp]
        L.conv_integer_forward.argtypes = [P, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp,
                                           ctypes.c_int, vp, vp]
        LP, GP, CP = (ctypes.POINTER(t) for t in (linear_problem, gated_problem, grad_clip_problem))
        for name, Q in (("linear", LP), ("linear_backward", LP), ("gated", GP),
                        ("gated_backward", GP)):
            getattr(L, name + "_scratch_size").argtypes = [Q, ctypes.c_int, u64p]
            getattr(L, name + "_describe_variant").argtypes = [Q, ctypes.c_int, ctypes.c_char_p,
                                                               ctypes.c_uint64]
        for name, Q, n in (("linear_check", LP, 7), ("linear_backward_check", LP, 9),
                           ("gated_check", GP, 9), ("gated_backward_check", GP, 12)):
            getattr(L, name).argtypes = [Q, ctypes.c_int] + [vp] * n + [ctypes.c_uint64]
        for name, Q, n in (("linear_forward", LP, 7), ("linear_backward", LP, 9),
                           ("gated_forward", GP, 9), ("gated_backward", GP, 12)):
            getattr(L, name).argtypes = [Q, ctypes.c_int] + [vp] * n + [ctypes.c_uint64, vp]
        L.grad_clip_scratch_size.argtypes = [CP, u64p]
        L.grad_clip_check.argtypes = [CP, vp, vp, ctypes.c_uint64]
        L.grad_clip.argtypes = [CP, vp, vp, ctypes.c_uint64, vp]
        L.conv_status_string.argtypes = [ctypes.c_int]
        L.conv_status_string.restype = ctypes.c_char_p
        for name in EXPORTS:
            getattr(L, name).restype = L.conv_status_string.restype if name == "conv_status_string" else ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().conv_status_string(int(status)).decode()


def make_problem(n, c_in, h, w, c_out, kh, kw, *, groups=1, stride=(1, 1), dilation=(1, 1),
                 pads=(0, 0, 0, 0), out_pad=(0, 0), transpose=False, act="identity",
                 alpha=None, beta=None, bias=False, residual=False, offsets=(0, 0, 0, 0, 0),
                 variant="auto", splits=0) -> conv_problem:
    """Fill a conv_problem; pads are (top, left, bottom, right)."""
    da, db = ACT_DEFAULTS.get(act, (0.0, 0.0))
    p = conv_problem()
    p.n, p.c_in, p.h, p.w, p.c_out, p.kh, p.kw = n, c_in, h, w, c_out, kh, kw
    p.groups = groups
    p.stride_h, p.stride_w = stride
    p.dil_h, p.dil_w = dilation
    p.pad_top, p.pad_left, p.pad_bottom, p.pad_right = pads
    p.out_pad_h, p.out_pad_w = out_pad
    p.x_off, p.w_off, p.b_off, p.r_off, p.y_off = offsets
    p.transpose = int(bool(transpose))
    p.activation = ACTIVATIONS[act]
    p.act_alpha = da if alpha is None else alpha
    p.act_beta = db if beta is None else beta
    p.has_bias = int(bool(bias))
    p.has_residual = int(bool(residual))
    p.variant_override = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    p.split_override = splits
    return p


def _dt(dtype):
    return DTYPES[dtype] if isinstance(dtype, str) else int(dtype)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def conv_output_extent(p: conv_problem):
    ho, wo = ctypes.c_int64(), ctypes.c_int64()
    st = lib().conv_output_extent(ctypes.byref(p), ctypes.byref(ho), ctypes.byref(wo))
    if st:
        raise ConvError(st, "conv_output_extent")
    return ho.value, wo.value


def conv_resolve_auto_pad(p: conv_problem, auto_pad, output_shape_hw=None) -> conv_problem:
    mode = AUTO_PAD[auto_pad] if isinstance(auto_pad, str) else int(auto_pad)
    arr = None
    if output_shape_hw is not None:
        arr = (ctypes.c_int64 * 2)(*output_shape_hw)
    st = lib().conv_resolve_auto_pad(ctypes.byref(p), mode, arr)
    if st:
        raise ConvError(st, "conv_resolve_auto_pad")
    return p


def conv_scratch_size(p: conv_problem, dtype):
    whole, per = ctypes.c_uint64(), ctypes.c_uint64()
    st = lib().conv_scratch_size(ctypes.byref(p), _dt(dtype), ctypes.byref(whole), ctypes.byref(per))
    if st:
        raise ConvError(st, "conv_scratch_size")
    return whole.value, per.value


def conv_describe_variant(p: conv_problem, dtype) -> str:
    buf = ctypes.create_string_buffer(256)
    st = lib().conv_describe_variant(ctypes.byref(p), _dt(dtype), buf, len(buf))
    if st:
        raise ConvError(st, "conv_describe_variant")
    return buf.value.decode()


def _call(fn, name, p, dtype, x, w, bias, residual, y, scratch, scratch_bytes, stream, check):
    st = fn(ctypes.byref(p), _dt(dtype), _ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y),
            _ptr(scratch), int(scratch_bytes), stream or None)
    if check and st:
        raise ConvError(st, name)
    return st


def conv_forward(p, dtype, x, w, bias, residual, y, scratch=None, scratch_bytes=0, stream=None,
                 check=True) -> int:
    """Enqueue the Conv forward on `stream` (a hipStream_t as int; None = default)."""
    return _call(lib().conv_forward, "conv_forward", p, dtype, x, w, bias, residual, y, scratch,
                 scratch_bytes, stream, check)


def conv_check(p, dtype, x, w, bias, residual, y, scratch=None, scratch_bytes=0) -> int:
    """Status conv_forward / conv_transpose_forward would return (host only)."""
    return lib().conv_check(ctypes.byref(p), _dt(dtype), _ptr(x), _ptr(w), _ptr(bias),
                            _ptr(residual), _ptr(y), _ptr(scratch), int(scratch_bytes))


def conv_transpose_forward(p, dtype, x, w, bias, residual, y, scratch=None, scratch_bytes=0,
                           stream=None, check=True) -> int:
    """Enqueue the ConvTranspose forward on `stream`."""
    return _call(lib().conv_transpose_forward, "conv_transpose_forward", p, dtype, x, w, bias,
                 residual, y, scratch, scratch_bytes, stream, check)


def conv_forward_noalloc(p, dtype, x, w, bias, residual, y, stream=None, check=True) -> int:
    """Enqueue Conv (p.transpose == 0) or ConvTranspose (p.transpose == 1) with the
    library's own static scratch: no allocation, no scratch argument."""
    st = lib().conv_forward_noalloc(ctypes.byref(p), _dt(dtype), _ptr(x), _ptr(w), _ptr(bias),
                                    _ptr(residual), _ptr(y), stream or None)
    if check and st:
        raise ConvError(st, "conv_forward_noalloc")
    return st


# ------------------------------------------------------------------ pooling

def make_pool_problem(n, c, h, w, kind="max", kernel=(1, 1), stride=(1, 1), dilation=(1, 1),
                      pads=(0, 0, 0, 0), ceil_mode=False, count_include_pad=False,
                      offsets=(0, 0)) -> pool_problem:
    """A pool_problem; pads are (top, left, bottom, right)."""
    return pool_problem(n, c, h, w, kernel[0], kernel[1], stride[0], stride[1], dilation[0],
                        dilation[1], pads[0], pads[1], pads[2], pads[3], offsets[0], offsets[1],
                        POOL_KINDS[kind] if isinstance(kind, str) else int(kind), int(ceil_mode),
                        int(count_include_pad), 0)


def pool_output_extent(p: pool_problem):
    ho, wo = ctypes.c_int64(), ctypes.c_int64()
    st = lib().pool_output_extent(ctypes.byref(p), ctypes.byref(ho), ctypes.byref(wo))
    if st:
        raise ConvError(st, "pool_output_extent")
    return ho.value, wo.value


def pool_resolve_auto_pad(p: pool_problem, auto_pad) -> pool_problem:
    mode = AUTO_PAD[auto_pad] if isinstance(auto_pad, str) else int(auto_pad)
    st = lib().pool_resolve_auto_pad(ctypes.byref(p), mode)
    if st:
        raise ConvError(st, "pool_resolve_auto_pad")
    return p


def pool_describe_variant(p: pool_problem, dtype) -> str:
    buf = ctypes.create_string_buffer(128)
    st = lib().pool_describe_variant(ctypes.byref(p), _dt(dtype), buf, len(buf))
    if st:
        raise ConvError(st, "pool_describe_variant")
    return buf.value.decode()


def pool_check(p: pool_problem, dtype, x, y) -> int:
    return lib().pool_check(ctypes.byref(p), _dt(dtype), _ptr(x), _ptr(y))


def pool_forward(p: pool_problem, dtype, x, y, stream=None, check=True) -> int:
    """Enqueue the pooling forward on `stream`."""
    st = lib().pool_forward(ctypes.byref(p), _dt(dtype), _ptr(x), _ptr(y), stream or None)
    if check and st:
        raise ConvError(st, "pool_forward")
    return st


# -------------------------------------------------------------- ConvInteger

CONVI_TYPES = {"u8": 0, "i8": 1}


def _it(t):
    return CONVI_TYPES[t] if isinstance(t, str) else int(t)


def conv_integer_describe_variant(p: conv_problem, x_type, w_type) -> str:
    buf = ctypes.create_string_buffer(128)
    st = lib().conv_integer_describe_variant(ctypes.byref(p), _it(x_type), _it(w_type), buf,
                                             len(buf))
    if st:
        raise ConvError(st, "conv_integer_describe_variant")
    return buf.value.decode()


def conv_integer_check(p, x_type, w_type, x, w, x_zero, w_zero, w_zero_per_channel, y) -> int:
    return lib().conv_integer_check(ctypes.byref(p), _it(x_type), _it(w_type), _ptr(x), _ptr(w),
                                    _ptr(x_zero), _ptr(w_zero), int(w_zero_per_channel), _ptr(y))


def conv_integer_forward(p, x_type, w_type, x, w, x_zero, w_zero, w_zero_per_channel, y,
                         stream=None, check=True) -> int:
    """Enqueue ConvInteger (int32 output with wrap-around) on `stream`."""
    st = lib().conv_integer_forward(ctypes.byref(p), _it(x_type), _it(w_type), _ptr(x), _ptr(w),
                                    _ptr(x_zero), _ptr(w_zero), int(w_zero_per_channel), _ptr(y),
                                    stream or None)
    if check and st:
        raise ConvError(st, "conv_integer_forward")
    return st


# ------------------------------------------- linear layer, gated feed-forward

# the activations of the linear and gated calls: the convolution's, and these
LINEAR_ACTIVATIONS = {**ACTIVATIONS, "gelu": 9, "gelu_tanh": 10}
RESIDUALS = {"none": 0, "before": 1, "after": 2}
W_LAYOUTS = {"nk": 0, "kn": 1}


def _code(table, v):
    return table[v] if isinstance(v, str) else int(v)


def make_linear_problem(m, n, k, *, act="identity", alpha=None, beta=None, bias=False,
                        residual="none", save_z=False, w_layout="nk", ldx=0, ldw=0, ldr=0, ldy=0,
                        ldz=0, lddx=0, lddw=0, lddr=0, offsets=(0, 0, 0, 0, 0, 0),
                        grad_offsets=(0, 0, 0, 0, 0)) -> linear_problem:
    """A linear_problem: y = act(x w^T + b [+ r]) [+ r], x [m, k], w [n, k] or [k, n].

    residual: "none", "before" or "after" the activation; ld*: row strides in
    elements (0 = dense); offsets: x, w, b, r, y, z; grad_offsets: dy, dx, dw, db, dr.
    """
    da, db = ACT_DEFAULTS.get(act, (0.0, 0.0))
    return linear_problem(m, n, k, ldx, ldw, ldr, ldy, ldz, lddx, lddw, lddr, *offsets,
                          *grad_offsets, _code(LINEAR_ACTIVATIONS, act),
                          da if alpha is None else alpha, db if beta is None else beta,
                          int(bias), _code(RESIDUALS, residual), int(save_z),
                          _code(W_LAYOUTS, w_layout), 0)


def make_gated_problem(m, f, k, *, act="silu", alpha=None, beta=None, bias=False, save=False,
                       ldx=0, ldw=0, ldh=0, ldp=0, lddx=0, lddw=0, offsets=(0,) * 8,
                       grad_offsets=(0,) * 6) -> gated_problem:
    """A gated_problem: h = act(x wg^T + bg) * (x wu^T + bu), x [m, k], wg, wu [f, k].

    save: the forward also stores both sums (pg, pu) for the backward pass;
    offsets: x, wg, wu, bg, bu, h, pg, pu; grad_offsets: dh, dx, dwg, dwu, dbg, dbu.
    """
    da, db = ACT_DEFAULTS.get(act, (0.0, 0.0))
    return gated_problem(m, f, k, ldx, ldw, ldh, ldp, lddx, lddw, *offsets, *grad_offsets,
                         _code(LINEAR_ACTIVATIONS, act), da if alpha is None else alpha,
                         db if beta is None else beta, int(bias), int(save), 0)


def _size(name, p, *dtype):
    n = ctypes.c_uint64()
    st = getattr(lib(), name)(ctypes.byref(p), *dtype, ctypes.byref(n))
    if st:
        raise ConvError(st, name)
    return n.value


def _describe(name, p, dtype):
    buf = ctypes.create_string_buffer(192)
    st = getattr(lib(), name)(ctypes.byref(p), _dt(dtype), buf, len(buf))
    if st:
        raise ConvError(st, name)
    return buf.value.decode()


def _run(name, p, dtype, operands, scratch, scratch_bytes, stream, check):
    st = getattr(_lib or lib(), name)(
        ctypes.byref(p), DTYPES[dtype] if isinstance(dtype, str) else int(dtype),
        *[t if t is None or isinstance(t, int) else t.data_ptr() for t in operands], _ptr(scratch),
        int(scratch_bytes), stream or None)
    if check and st:
        raise ConvError(st, name)
    return st


def linear_scratch_size(p: linear_problem, dtype) -> int:
    return _size("linear_scratch_size", p, _dt(dtype))


def linear_backward_scratch_size(p: linear_problem, dtype) -> int:
    return _size("linear_backward_scratch_size", p, _dt(dtype))


def linear_describe_variant(p: linear_problem, dtype) -> str:
    return _describe("linear_describe_variant", p, dtype)


def linear_backward_describe_variant(p: linear_problem, dtype) -> str:
    return _describe("linear_backward_describe_variant", p, dtype)


def linear_check(p, dtype, x, w, b, r, y, z=None, scratch=None, scratch_bytes=0) -> int:
    """Status linear_forward would return before enqueueing (host only)."""
    return lib().linear_check(ctypes.byref(p), _dt(dtype), _ptr(x), _ptr(w), _ptr(b), _ptr(r),
                              _ptr(y), _ptr(z), _ptr(scratch), int(scratch_bytes))


def linear_backward_check(p, dtype, x, w, z, dy, dx, dw, db, dr, scratch=None,
                          scratch_bytes=0) -> int:
    return lib().linear_backward_check(ctypes.byref(p), _dt(dtype),
                                       *map(_ptr, (x, w, z, dy, dx, dw, db, dr)), _ptr(scratch),
                                       int(scratch_bytes))


def linear_forward(p, dtype, x, w, b, r, y, z=None, scratch=None, scratch_bytes=0, stream=None,
                   check=True) -> int:
    """Enqueue the linear layer on `stream`; z receives the sums before the
    activation when the problem asks for them (save_z)."""
    return _run("linear_forward", p, dtype, (x, w, b, r, y, z), scratch, scratch_bytes, stream,
                check)


def linear_backward(p, dtype, x, w, z, dy, dx, dw, db, dr, scratch=None, scratch_bytes=0,
                    stream=None, check=True) -> int:
    """Enqueue the gradients of the linear layer; those passed as None are not computed."""
    return _run("linear_backward", p, dtype, (x, w, z, dy, dx, dw, db, dr), scratch,
                scratch_bytes, stream, check)


def gated_scratch_size(p: gated_problem, dtype) -> int:
    return _size("gated_scratch_size", p, _dt(dtype))


def gated_backward_scratch_size(p: gated_problem, dtype) -> int:
    return _size("gated_backward_scratch_size", p, _dt(dtype))


def gated_describe_variant(p: gated_problem, dtype) -> str:
    return _describe("gated_describe_variant", p, dtype)


def gated_backward_describe_variant(p: gated_problem, dtype) -> str:
    return _describe("gated_backward_describe_variant", p, dtype)


def gated_check(p, dtype, x, wg, wu, bg, bu, h, pg=None, pu=None, scratch=None,
                scratch_bytes=0) -> int:
    """Status gated_forward would return before enqueueing (host only)."""
    return lib().gated_check(ctypes.byref(p), _dt(dtype),
                             *map(_ptr, (x, wg, wu, bg, bu, h, pg, pu)), _ptr(scratch),
                             int(scratch_bytes))


def gated_backward_check(p, dtype, x, wg, wu, pg, pu, dh, dx, dwg, dwu, dbg, dbu, scratch=None,
                         scratch_bytes=0) -> int:
    return lib().gated_backward_check(ctypes.byref(p), _dt(dtype),
                                      *map(_ptr, (x, wg, wu, pg, pu, dh, dx, dwg, dwu, dbg, dbu)),
                                      _ptr(scratch), int(scratch_bytes))


def gated_forward(p, dtype, x, wg, wu, bg, bu, h, pg=None, pu=None, scratch=None, scratch_bytes=0,
                  stream=None, check=True) -> int:
    """Enqueue the gated projection on `stream`; pg and pu receive both sums when
    the problem asks for them (save)."""
    return _run("gated_forward", p, dtype, (x, wg, wu, bg, bu, h, pg, pu), scratch, scratch_bytes,
                stream, check)


def gated_backward(p, dtype, x, wg, wu, pg, pu, dh, dx, dwg, dwu, dbg, dbu, scratch=None,
                   scratch_bytes=0, stream=None, check=True) -> int:
    """Enqueue the gradients of the gated projection; those passed as None are not
    computed (dwg and dwu, dbg and dbu go in pairs)."""
    return _run("gated_backward", p, dtype, (x, wg, wu, pg, pu, dh, dx, dwg, dwu, dbg, dbu),
                scratch, scratch_bytes, stream, check)


# ------------------------------------------------------------ gradient clipping

NORMS = {1: 1, 2: 2, float("inf"): 3}


def make_grad_clip_problem(grads, outs, dtype, *, norm=2, max_norm=1.0, eps=1e-6,
                           elems=None) -> grad_clip_problem:
    """The table of a grad_clip call.

    grads: contiguous tensors, or device pointers with their lengths in elems;
    outs: where the clipped gradients go (the gradients themselves clip in
    place), or None for the norm alone; dtype: one for all, or one each;
    norm: 1, 2 or inf.  The problem holds the pointers, not the tensors.
    """
    n = len(grads)
    table = (grad_tensor * max(n, 1))()
    for i, g in enumerate(grads):
        if elems is None and not g.is_contiguous():
            raise ValueError(f"gradient {i} is not contiguous")
        if outs is not None and elems is None and (
                not outs[i].is_contiguous() or outs[i].numel() != g.numel()):
            raise ValueError(f"output {i} is not contiguous or of another length")
        table[i] = grad_tensor(_ptr(g), None if outs is None else _ptr(outs[i]),
                               g.numel() if elems is None else elems[i],
                               _dt(dtype if isinstance(dtype, (str, int)) else dtype[i]), 0)
    return grad_clip_problem(table, n, NORMS[norm], max_norm, eps, 0)


def grad_clip_scratch_size(p: grad_clip_problem) -> int:
    return _size("grad_clip_scratch_size", p)


def grad_clip_check(p: grad_clip_problem, norm, scratch=None, scratch_bytes=0) -> int:
    """Status grad_clip would return before enqueueing (host only)."""
    return lib().grad_clip_check(ctypes.byref(p), _ptr(norm), _ptr(scratch), int(scratch_bytes))


def grad_clip(p: grad_clip_problem, norm, scratch=None, scratch_bytes=0, stream=None,
              check=True) -> int:
    """Enqueue the global norm (into norm, one float32) and the clipping on `stream`."""
    st = lib().grad_clip(ctypes.byref(p), _ptr(norm), _ptr(scratch), int(scratch_bytes),
                         stream or None)
    if check and st:
        raise ConvError(st, "grad_clip")
    return st
