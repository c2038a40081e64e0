"""ctypes binding of the FFN sub-layer's operators in libgemm_rs.so: the
block norm (include/block_norm.h), the 8-bit integer product
(include/gemm_q8.h), the products grouped by expert (include/gemm_grouped.h),
and the dense products: the gated projections (include/gemm_gated.h) and the
product with bias, activation and residual (include/gemm_epi.h).

Argument marshalling only, as in ``gemm_rs``: tensors go in as device
pointers, the stream as its ``hipStream_t`` handle, and a non-OK status
raises ``GemmRsError`` from the owning wrappers.  The plans of the dense
products, whose arrays have types and strides of their own, refuse tensors
that do not hold what the plan takes them for; addresses are taken as they are.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

from .gemm_rs import (BF16, ERR_HIP, ERR_INVALID_ARG, ERR_PROTOCOL, ERR_UNSUPPORTED, F32, OK,
                      GemmRsError, _stream_handle, gemm_rs_strerror, load_library)

__all__ = ["BF16", "F32", "OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED", "ERR_HIP", "ERR_PROTOCOL",
           "GROUPED_NN", "GROUPED_NT", "GROUPED_TN", "GemmRsError", "gemm_rs_strerror",
           "WEIGHTS_KN", "WEIGHTS_NK", "ACT_NONE", "ACT_RELU", "ACT_GELU", "ACT_GELU_TANH", "ACT_SILU",
           "BlockNormPlan", "Q8Plan", "GroupedPlan", "GatedPlan", "EpiPlan", "q8_quantize"]

_INC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
HEADERS = [os.path.join(_INC, h) for h in ("block_norm.h", "gemm_q8.h", "gemm_grouped.h")]
DENSE_HEADERS = [os.path.join(_INC, h) for h in ("gemm_gated.h", "gemm_epi.h")]

GROUPED_NN, GROUPED_NT, GROUPED_TN = 0, 1, 2
WEIGHTS_KN, WEIGHTS_NK = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4


class block_norm_desc_t(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("stream_dtype", ctypes.c_int32),
        ("param_dtype", ctypes.c_int32), ("has_y", ctypes.c_int32),
        ("post", ctypes.c_int32), ("pre", ctypes.c_int32),
        ("quant", ctypes.c_int32), ("backward", ctypes.c_int32),
        ("rows_per_gate", ctypes.c_int64),
        ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64),
        ("ld_x_out", ctypes.c_int64), ("ld_u", ctypes.c_int64),
        ("ld_dx_out", ctypes.c_int64), ("ld_du", ctypes.c_int64),
        ("ld_dx", ctypes.c_int64), ("ld_dy", ctypes.c_int64),
        ("res_scale", ctypes.c_float), ("weight_offset", ctypes.c_float),
        ("eps_post", ctypes.c_float), ("eps_pre", ctypes.c_float),
        ("pad", ctypes.c_int32),
    ]


class block_norm_info_t(ctypes.Structure):
    _fields_ = [("gate_rows", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64)]


class gemm_q8_desc_t(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("lda", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldd", ctypes.c_int64),
        ("out_dtype", ctypes.c_int32), ("has_bias", ctypes.c_int32),
    ]


class gemm_q8_info_t(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64)]


class gemm_grouped_desc_t(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("E", ctypes.c_int32), ("op", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32),
        ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64),
        ("pad", ctypes.c_int64),
    ]


class gemm_grouped_info_t(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64)]


class gemm_gated_desc_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("M", "N", "K")] +
                [(n, ctypes.c_int32) for n in ("layout", "act", "has_bias", "bias_dtype", "backward",
                                               "dw_dtype", "accumulate", "z_dtype")] +
                [(n, ctypes.c_int64) for n in ("ldx", "ldw", "ldh", "ldz", "lddh", "lddz", "lddx", "lddw")])


class gemm_gated_info_t(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64)]


class gemm_epi_desc_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("M", "N", "K")] +
                [(n, ctypes.c_int32) for n in ("layout", "act", "out_dtype", "has_bias", "bias_dtype",
                                               "has_residual", "backward", "dw_dtype", "accumulate", "z_dtype")] +
                [(n, ctypes.c_int64) for n in ("ldx", "ldw", "ldr", "ldy", "ldz", "lddy", "lddz", "lddx", "lddw")])


class gemm_epi_info_t(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64)]


_lib = None


def _library() -> ctypes.CDLL:
    """The HIP library with these entry points' types set (once)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = load_library()
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    ptr = ctypes.POINTER
    types = {
        "block_norm_plan": [ptr(block_norm_desc_t), ptr(vp)],
        "block_norm_run": [vp] * 9 + [i64, vp],
        "block_norm_backward": [vp] * 13 + [i64, vp],
        "block_norm_query": [vp, ptr(block_norm_info_t)],
        "block_norm_destroy": [vp],
        "gemm_q8_plan": [ptr(gemm_q8_desc_t), ptr(vp)],
        "gemm_q8_run": [vp] * 7 + [i64, vp],
        "gemm_q8_quantize": [vp, i32, i64, i64, i64, vp, i64, vp, vp],
        "gemm_q8_query": [vp, ptr(gemm_q8_info_t)],
        "gemm_q8_destroy": [vp],
        "gemm_grouped_plan": [ptr(gemm_grouped_desc_t), ptr(vp)],
        "gemm_grouped_run": [vp] * 5 + [i64, vp],
        "gemm_grouped_status": [vp, vp, ptr(i32)],
        "gemm_grouped_query": [vp, ptr(gemm_grouped_info_t)],
        "gemm_grouped_destroy": [vp],
        "gemm_gated_plan": [ptr(gemm_gated_desc_t), ptr(vp)],
        "gemm_gated_run": [vp] * 9 + [i64, vp],
        "gemm_gated_backward": [vp] * 14 + [i64, vp],
        "gemm_gated_query": [vp, ptr(gemm_gated_info_t)],
        "gemm_gated_destroy": [vp],
        "gemm_epi_plan": [ptr(gemm_epi_desc_t), ptr(vp)],
        "gemm_epi_run": [vp] * 7 + [i64, vp],
        "gemm_epi_backward": [vp] * 9 + [i64, vp],
        "gemm_epi_query": [vp, ptr(gemm_epi_info_t)],
        "gemm_epi_destroy": [vp],
    }
    for name, args in types.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ctypes.c_int
    _lib = lib
    return lib


def header_functions(paths=None):
    """Names of the functions these headers declare."""
    names = set()
    for path in paths or HEADERS:
        text = open(path).read()
        names.update(re.findall(r"GEMM_RS_API\s+[\w\s\*]+?\b((?:block_norm|gemm_q8|gemm_grouped|"
                                r"gemm_gated|gemm_epi)_\w+)\s*\(", text))
    return sorted(names)


def _check(rc: int, where: str) -> None:
    if rc != OK:
        raise GemmRsError(rc, where)


def _addresses(*tensors):
    """Device addresses of tensors (or addresses, or None), as `_ptr` of each:
    one pass, since a call on few tokens takes less time than its marshalling."""
    return [t if t is None or t.__class__ is int else t.data_ptr() for t in tensors]


def _check_offsets(t, n):
    """Refuses a tensor that does not hold n int32 one after another on the GPU:
    the kernels would take its bits for offsets, and most would pass for valid
    ones (int64, the default of cumsum, reads as 0 every other time)."""
    if t.element_size() != 4 or t.is_floating_point() or t.numel() < n or not (t.is_cuda and t.is_contiguous()):
        raise GemmRsError(ERR_INVALID_ARG, "gemm_grouped_run: offsets are not %d contiguous int32 on the GPU" % n)


def _holds(t, rows, cols, ld):
    """Whether a tensor's elements lie as `rows` rows of `cols`, ld elements apart."""
    shape, stride = t.shape, t.stride()
    if not shape:
        return rows * cols <= 1
    if len(shape) == 2 and stride == (ld, 1) and shape[0] >= rows and shape[1] >= cols:
        return True
    if shape[-1] > 1 and stride[-1] != 1:
        return False
    have = 1                        # rows of the tensor, equally far apart
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] > 1 and stride[i] != ld * have:
            return False
        have *= shape[i]
    if have >= rows and shape[-1] >= cols:
        return True
    return t.is_contiguous() and t.numel() >= (rows - 1) * ld + cols       # (an array without a shape of its own)


class _Plan:
    """Owns one plan handle of the family `_name`."""

    _name = ""
    _info_t = None

    def __init__(self, desc):
        self.handle = None
        self.desc = desc
        self._lib = _library()
        h = ctypes.c_void_p()
        _check(getattr(self._lib, self._name + "_plan")(ctypes.byref(desc), ctypes.byref(h)),
               self._name + "_plan")
        self.handle = h.value
        self._run = getattr(self._lib, self._name + "_run")

    @property
    def info(self):
        info = self._info_t()
        _check(getattr(self._lib, self._name + "_query")(self.handle, ctypes.byref(info)),
               self._name + "_query")
        return info

    def close(self):
        if self.handle is not None:
            getattr(self._lib, self._name + "_destroy")(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BlockNormPlan(_Plan):
    """Norms before and after a block with gate and residual scale."""

    _name, _info_t = "block_norm", block_norm_info_t

    def __init__(self, rows, cols, dtype=BF16, stream_dtype=BF16, param_dtype=F32, has_y=1, post=1,
                 pre=1, quant=0, backward=0, rows_per_gate=0, res_scale=1.0, weight_offset=0.0,
                 eps_post=1e-6, eps_pre=1e-6, **strides):
        super().__init__(block_norm_desc_t(
            rows=rows, cols=cols, dtype=dtype, stream_dtype=stream_dtype, param_dtype=param_dtype,
            has_y=has_y, post=post, pre=pre, quant=quant, backward=backward,
            rows_per_gate=rows_per_gate, res_scale=res_scale, weight_offset=weight_offset,
            eps_post=eps_post, eps_pre=eps_pre, **strides))
        self._rows = rows

    def run(self, x, y, w_post, gate, w_pre, x_out, u, u_scale=None, rows=None, stream=None):
        rc = self._run(self.handle, *_addresses(x, y, w_post, gate, w_pre, x_out, u, u_scale),
                       self._rows if rows is None else rows, _stream_handle(stream))
        if rc != OK:
            raise GemmRsError(rc, "block_norm_run")

    def backward(self, dx_out, du, x_out, y, w_post, gate, w_pre, dx, dy, dw_post, dgate, dw_pre,
                 rows=None, stream=None):
        _check(self._lib.block_norm_backward(
            self.handle, *_addresses(dx_out, du, x_out, y, w_post, gate, w_pre, dx, dy, dw_post,
                                     dgate, dw_pre),
            self._rows if rows is None else rows, _stream_handle(stream)), "block_norm_backward")


class Q8Plan(_Plan):
    """8-bit integer product with scales per token and per channel."""

    _name, _info_t = "gemm_q8", gemm_q8_info_t

    def __init__(self, M, N, K, lda=0, ldw=0, ldd=0, out_dtype=BF16, has_bias=0):
        super().__init__(gemm_q8_desc_t(M=M, N=N, K=K, lda=lda, ldw=ldw, ldd=ldd,
                                        out_dtype=out_dtype, has_bias=has_bias))
        self._rows = M

    def run(self, a, a_scale, w, w_scale, bias, D, rows=None, stream=None):
        rc = self._run(self.handle, *_addresses(a, a_scale, w, w_scale, bias, D),
                       self._rows if rows is None else rows, _stream_handle(stream))
        if rc != OK:
            raise GemmRsError(rc, "gemm_q8_run")


def q8_quantize(x, q, scale, rows, cols, dtype=BF16, ldx=0, ldq=0, stream=None) -> None:
    """Rows of x to int8 rows and one scale per row (strides 0: tight, the
    int8 rows up to a multiple of 16)."""
    x, q, scale = _addresses(x, q, scale)
    rc = (_lib or _library()).gemm_q8_quantize(x, dtype, rows, cols, ldx or cols, q,
                                               ldq or (cols + 15) // 16 * 16, scale,
                                               _stream_handle(stream))
    if rc != OK:
        raise GemmRsError(rc, "gemm_q8_quantize")


class GroupedPlan(_Plan):
    """Products grouped by expert with ragged group sizes."""

    _name, _info_t = "gemm_grouped", gemm_grouped_info_t

    def __init__(self, M, N, K, E, op, out_dtype=BF16, accumulate=0, lda=0, ldb=0, ldc=0):
        super().__init__(gemm_grouped_desc_t(M=M, N=N, K=K, E=E, op=op, out_dtype=out_dtype,
                                             accumulate=accumulate, lda=lda, ldb=ldb, ldc=ldc))
        self._rows = M
        self._offsets = E + 1

    def run(self, A, B, offsets, C, rows=None, stream=None):
        """offsets: an int32 tensor of E + 1 on the GPU, or an address."""
        if hasattr(offsets, "element_size"):        # (neither an address nor a bare data_ptr())
            _check_offsets(offsets, self._offsets)
        rc = self._run(self.handle, *_addresses(A, B, offsets, C),
                       self._rows if rows is None else rows, _stream_handle(stream))
        if rc != OK:
            raise GemmRsError(rc, "gemm_grouped_run")

    def status(self, stream=None):
        """Returns (status, [code, expert, offsets[e], offsets[e+1]])."""
        detail = (ctypes.c_int32 * 4)()
        rc = self._lib.gemm_grouped_status(self.handle, _stream_handle(stream), detail)
        return rc, list(detail)


class _DensePlan(_Plan):
    """A plan that knows its arrays: their types, rows (None: a call's), columns and strides."""

    def __init__(self, desc):
        super().__init__(desc)
        self._rows = desc.M
        self._w = (desc.K, desc.N) if desc.layout == WEIGHTS_KN else (desc.N, desc.K)
        self._tensor, self._types, self._device = (), {}, 0
        try:
            import torch
        except ImportError:            # (then arrays are addresses)
            return
        self._tensor = torch.Tensor
        self._types = {BF16: (torch.bfloat16, torch.int16, torch.uint16), F32: (torch.float32,)}      # (bfloat16 may come as its bits)
        if torch.cuda.is_available():
            self._device = torch.cuda.current_device()

    def _array(self, name, dtype, rows, cols, ld):
        types = self._types.get(dtype, (None,))
        # (with the shape that most calls bring, where tight rows are the plan's)
        return types[0], (self._rows if rows is None else rows, cols) if ld in (0, cols) else None, (name, types, rows, cols, ld or cols)

    def _arrays(self, where, arrays, tensors, rows):
        """Device addresses of tensors, as `_addresses`.  The kernels know an array by
        its address alone: one of another type, length or stride, of the host's or of
        another device would be read and written past its end, so it is refused.
        It costs 0.3 us an array on the host: one row of 256 x 256, four arrays, takes
        5.0 us a call instead of 3.7; one of 3584 x 8192 takes the GPU's 10.3 either way."""
        T, device = self._tensor, self._device
        return [t if t is None or t.__class__ is int else
                t.data_ptr() if isinstance(t, T) and t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous() else
                self._address(where, array, t, rows) for t, (dtype, shape, array) in zip(tensors, arrays)]

    def _address(self, where, array, t, rows):
        name, types, n, cols, ld = array
        if isinstance(t, self._tensor):            # (else anything that has an address)
            if n is None:
                n = rows
            if t.dtype not in types or t.get_device() != self._device or not (n <= 0 or _holds(t, n, cols, ld)):
                raise GemmRsError(ERR_INVALID_ARG, "%s: %s (%s, shape %s, stride %s, %s) is not %d x %d of %s, rows %d apart, on GPU %d" % (
                    where, name, t.dtype, tuple(t.shape), t.stride(), t.device, n, cols, types[0], ld, self._device))
        return t.data_ptr()


class GatedPlan(_DensePlan):
    """Gated projections, h = act(x w_gate + b_gate) * (x w_up + b_up), and their backward pass."""

    _name, _info_t = "gemm_gated", gemm_gated_info_t

    def __init__(self, M, N, K, layout=WEIGHTS_KN, act=ACT_SILU, has_bias=0, bias_dtype=F32, backward=0,
                 dw_dtype=BF16, accumulate=0, z_dtype=BF16, **strides):
        super().__init__(gemm_gated_desc_t(M=M, N=N, K=K, layout=layout, act=act, has_bias=has_bias,
                                           bias_dtype=bias_dtype, backward=backward, dw_dtype=dw_dtype,
                                           accumulate=accumulate, z_dtype=z_dtype, **strides))
        d, a = self.desc, self._array
        x, w = a("x", BF16, None, K, d.ldx), [a("w_" + k, BF16, *self._w, d.ldw) for k in ("gate", "up")]
        z = [a("z_" + k, z_dtype, None, N, d.ldz) for k in ("gate", "up")]
        self._forward = [x, *w, *(a("b_" + k, bias_dtype, 1, N, 0) for k in ("gate", "up")), a("h", BF16, None, N, d.ldh), *z]
        self._backward = [a("dh", BF16, None, N, d.lddh), x, *w, *z, *(a("dz_" + k, BF16, None, N, d.lddz) for k in ("gate", "up")),
                          a("dx", BF16, None, K, d.lddx), *(a("dw_" + k, dw_dtype, *self._w, d.lddw) for k in ("gate", "up")),
                          *(a("db_" + k, F32, 1, N, 0) for k in ("gate", "up"))]

    def run(self, x, w_gate, w_up, b_gate, b_up, h, z_gate=None, z_up=None, rows=None, stream=None):
        rows = self._rows if rows is None else rows
        rc = self._run(self.handle, *self._arrays("gemm_gated_run", self._forward, (x, w_gate, w_up, b_gate, b_up, h, z_gate, z_up), rows),
                       rows, _stream_handle(stream))
        if rc != OK:
            raise GemmRsError(rc, "gemm_gated_run")

    def backward(self, dh, x, w_gate, w_up, z_gate, z_up, dz_gate, dz_up, dx, dw_gate=None, dw_up=None,
                 db_gate=None, db_up=None, rows=None, stream=None):
        rows = self._rows if rows is None else rows
        _check(self._lib.gemm_gated_backward(
            self.handle, *self._arrays("gemm_gated_backward", self._backward,
                                       (dh, x, w_gate, w_up, z_gate, z_up, dz_gate, dz_up, dx, dw_gate, dw_up, db_gate, db_up), rows),
            rows, _stream_handle(stream)), "gemm_gated_backward")


class EpiPlan(_DensePlan):
    """Product with bias, activation and residual, y = act(x w + bias) + r, and its backward pass."""

    _name, _info_t = "gemm_epi", gemm_epi_info_t

    def __init__(self, M, N, K, layout=WEIGHTS_KN, act=ACT_NONE, out_dtype=BF16, has_bias=0, bias_dtype=F32,
                 has_residual=0, backward=0, dw_dtype=BF16, accumulate=0, z_dtype=BF16, **strides):
        super().__init__(gemm_epi_desc_t(M=M, N=N, K=K, layout=layout, act=act, out_dtype=out_dtype,
                                         has_bias=has_bias, bias_dtype=bias_dtype, has_residual=has_residual,
                                         backward=backward, dw_dtype=dw_dtype, accumulate=accumulate,
                                         z_dtype=z_dtype, **strides))
        d, a = self.desc, self._array
        x, w, z = a("x", BF16, None, K, d.ldx), a("w", BF16, *self._w, d.ldw), a("z", z_dtype, None, N, d.ldz)
        self._forward = [x, w, a("bias", bias_dtype, 1, N, 0), a("r", out_dtype, None, N, d.ldr), a("y", out_dtype, None, N, d.ldy), z]
        self._backward = [a("dy", out_dtype, None, N, d.lddy), x, w, z, a("dz", BF16, None, N, d.lddz), a("dx", BF16, None, K, d.lddx),
                          a("dw", dw_dtype, *self._w, d.lddw), a("dbias", F32, 1, N, 0)]

    def run(self, x, w, bias, r, y, z=None, rows=None, stream=None):
        rows = self._rows if rows is None else rows
        rc = self._run(self.handle, *self._arrays("gemm_epi_run", self._forward, (x, w, bias, r, y, z), rows), rows, _stream_handle(stream))
        if rc != OK:
            raise GemmRsError(rc, "gemm_epi_run")

    def backward(self, dy, x, w, z, dz, dx, dw=None, dbias=None, rows=None, stream=None):
        rows = self._rows if rows is None else rows
        _check(self._lib.gemm_epi_backward(
            self.handle, *self._arrays("gemm_epi_backward", self._backward, (dy, x, w, z, dz, dx, dw, dbias), rows),
            rows, _stream_handle(stream)), "gemm_epi_backward")
