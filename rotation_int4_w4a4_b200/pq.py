"""ctypes binding for libpq (``include/pq.h``): the same entry points, argument marshalling only.

Tensors are passed as device pointers (``torch.Tensor.data_ptr()``) with the current CUDA
stream unless one is given.  Every call checks the returned status and raises ``PQError``
with the library's message.  Importing this module loads the library and raises if it has
not been built (``python -m rotation_int4_w4a4_b200.build``): there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import warnings

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libpq.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libpq.so is not built ({_LIB_PATH}); run python -m rotation_int4_w4a4_b200.build")
lib = ctypes.CDLL(_LIB_PATH)

PQ_OK, PQ_ERR_INVALID_ARG, PQ_ERR_UNSUPPORTED, PQ_ERR_CUDA, PQ_ERR_ALLOC, PQ_ERR_TIMEOUT = range(6)
PQ_HADAMARD, PQ_GIVENS, PQ_SMOOTH_HADAMARD = range(3)
PQ_OUT_F32, PQ_OUT_BF16 = range(2)
PQ_FLAG_SMOOTH_AFTER_ROTATE = 0x1
PQ_NO_PAIR = 0xFF
PQ_KV4_ROTATE_K, PQ_KV4_ROTATE_V = 0x1, 0x2
PQ_KV4_INTERLEAVED = 0x1
PQ_FP4_MX, PQ_FP4_NV = range(2)
FP4_FORMATS = {"mx": PQ_FP4_MX, "nv": PQ_FP4_NV}
KINDS = {"hadamard": PQ_HADAMARD, "givens": PQ_GIVENS, "smooth_hadamard": PQ_SMOOTH_HADAMARD}

# Every symbol the header declares.
EXPORTS = ("pq_select_pairs", "pq_make_plan", "pq_destroy_plan", "pq_transform_quant",
           "pq_pack_weights", "pq_w4a4_gemm", "pq_w4a4_gemm_noalloc", "pq_w4a4_gemm_launch_count",
           "pq_w4a4_gemm_launch_count_g", "pq_w4a4_linear", "pq_make_plan_outliers",
           "pq_rrs_prepare", "pq_rrs_transform_quant", "pq_rrs_pack_weights", "pq_rrs_gemm",
           "pq_quant_rows8", "pq_w8a8_gemm", "pq_w8a8_linear",
           "pq_fp4_scale_bytes", "pq_quant_fp4", "pq_fp4_gemm", "pq_fp4_linear",
           "pq_kv4_append", "pq_kv4_read", "pq_kv4_attention", "pq_kv4_attention_masked",
           "pq_check_status",
           "pq_selftest_wait_timeout", "pq_status_string", "pq_last_error")

_c = ctypes
_vp, _i64, _u64, _i32, _u32 = _c.c_void_p, _c.c_int64, _c.c_uint64, _c.c_int, _c.c_uint32
lib.pq_select_pairs.argtypes = [_u64, _i32, _i32, _i32, _i32, _vp]
lib.pq_select_pairs.restype = _i32
lib.pq_make_plan.argtypes = [_c.POINTER(_vp), _i32, _i32, _i32, _i32, _vp, _vp, _vp, _u32]
lib.pq_make_plan.restype = _i32
lib.pq_make_plan_outliers.argtypes = [_c.POINTER(_vp), _i32, _i32, _i32, _i32, _vp, _vp, _vp, _u32, _i32, _vp]
lib.pq_make_plan_outliers.restype = _i32
lib.pq_destroy_plan.argtypes = [_vp]
lib.pq_destroy_plan.restype = None
lib.pq_transform_quant.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]
lib.pq_transform_quant.restype = _i32
lib.pq_pack_weights.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp]
lib.pq_pack_weights.restype = _i32
lib.pq_w4a4_gemm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _i32, _vp]
lib.pq_w4a4_gemm.restype = _i32
lib.pq_w4a4_gemm_noalloc.argtypes = lib.pq_w4a4_gemm.argtypes
lib.pq_w4a4_gemm_noalloc.restype = _i32
lib.pq_w4a4_gemm_launch_count.argtypes = [_i64, _i64, _i64, _c.POINTER(_i32)]
lib.pq_w4a4_gemm_launch_count.restype = _i32
lib.pq_w4a4_gemm_launch_count_g.argtypes = [_i64, _i64, _i64, _i32, _c.POINTER(_i32)]
lib.pq_w4a4_gemm_launch_count_g.restype = _i32
lib.pq_w4a4_linear.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _i32, _vp]
lib.pq_w4a4_linear.restype = _i32
lib.pq_rrs_prepare.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]
lib.pq_rrs_prepare.restype = _i32
lib.pq_rrs_transform_quant.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]
lib.pq_rrs_transform_quant.restype = _i32
lib.pq_rrs_pack_weights.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp]
lib.pq_rrs_pack_weights.restype = _i32
lib.pq_rrs_gemm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _i32, _vp]
lib.pq_rrs_gemm.restype = _i32
_f32 = _c.c_float
lib.pq_quant_rows8.argtypes = [_vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp]
lib.pq_quant_rows8.restype = _i32
lib.pq_w8a8_gemm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp]
lib.pq_w8a8_gemm.restype = _i32
lib.pq_w8a8_linear.argtypes = [_vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _i32, _vp]
lib.pq_w8a8_linear.restype = _i32
lib.pq_fp4_scale_bytes.argtypes = [_i64, _i64, _i32]
lib.pq_fp4_scale_bytes.restype = _i64
lib.pq_quant_fp4.argtypes = [_vp, _i64, _i64, _i64, _i32, _i32, _f32, _vp, _vp, _vp]
lib.pq_quant_fp4.restype = _i32
lib.pq_fp4_gemm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _f32, _vp, _i32, _vp]
lib.pq_fp4_gemm.restype = _i32
lib.pq_fp4_linear.argtypes = [_vp, _i64, _i64, _i64, _i32, _i32, _f32, _vp, _vp, _vp, _vp, _f32, _i64, _vp, _i32, _vp]
lib.pq_fp4_linear.restype = _i32


class _KV4Struct(_c.Structure):
    _fields_ = [("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp), ("pages", _i64),
                ("page_size", _c.c_int32), ("heads", _c.c_int32), ("head_dim", _c.c_int32), ("flags", _u32)]


lib.pq_kv4_append.argtypes = [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _vp, _f32, _vp, _i64, _i32, _vp,
                              _vp, _u32, _vp, _vp]
lib.pq_kv4_append.restype = _i32
lib.pq_kv4_read.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp]
lib.pq_kv4_read.restype = _i32
lib.pq_kv4_attention.argtypes = [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _f32, _i64, _vp,
                                 _i64, _vp]
lib.pq_kv4_attention.restype = _i32
lib.pq_kv4_attention_masked.argtypes = [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _f32, _i64, _i64,
                                        _vp, _i64, _vp, _i64, _vp]
lib.pq_kv4_attention_masked.restype = _i32
lib.pq_selftest_wait_timeout.argtypes = [_u64, _vp]
lib.pq_selftest_wait_timeout.restype = _i32
lib.pq_check_status.argtypes = [_vp, _vp]
lib.pq_check_status.restype = _i32
lib.pq_status_string.argtypes = [_i32]
lib.pq_status_string.restype = _c.c_char_p
lib.pq_last_error.argtypes = []
lib.pq_last_error.restype = _c.c_char_p


class PQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.pq_last_error().decode(errors="replace")
        super().__init__(f"{where}: {lib.pq_status_string(status).decode()}: {msg}")


def _check(status: int, where: str) -> None:
    if status != PQ_OK:
        raise PQError(status, where)


def _ptr(x, rows_strided=False):
    """Device pointer of a tensor (None -> NULL; an int passes through as a raw address).

    The library reads and writes dense row-major device buffers, so a tensor must live on a
    CUDA device and be contiguous; with rows_strided (the activations, whose row stride is
    passed as ldx) only the last dimension must be contiguous.  Anything else would be read at
    the wrong addresses, so it is rejected here instead.
    """
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not getattr(x, "is_cuda", False):
        raise ValueError("expected a CUDA tensor: the library takes device pointers")
    if not (x.stride(-1) == 1 if rows_strided else x.is_contiguous()):
        raise ValueError("expected a contiguous tensor" + (" along its last dimension" if rows_strided else ""))
    return x.data_ptr()


def _arg(x, name, dtype, need, rows_strided=False):
    """Pointer of a tensor argument after checking its dtype and that it holds at least `need`
    elements (the C ABI only sees a pointer: a wrong dtype or a short buffer would make the
    kernels read or write past its end).  Raw integer addresses pass unchecked."""
    if x is None or isinstance(x, int):
        return _ptr(x)
    import torch
    want = {"bf16": (torch.bfloat16,), "u8": (torch.uint8,), "i8": (torch.int8,), "f32": (torch.float32,),
            "i32": (torch.int32,), "i64": (torch.int64,), "y": (torch.float32, torch.bfloat16)}[dtype]
    if x.dtype not in want:
        raise ValueError(f"{name}: dtype {x.dtype} is not accepted (expected {' or '.join(map(str, want))})")
    p = _ptr(x, rows_strided)
    if rows_strided:
        if x.dim() != 2:
            raise ValueError(f"{name}: expected a 2-D tensor")
        extent = (x.shape[0] - 1) * x.stride(0) + x.shape[1] if x.shape[0] > 0 else 0
    else:
        extent = x.numel()
    if extent < need:
        raise ValueError(f"{name}: holds {extent} elements, the call needs {need}")
    return p


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def pq_select_pairs(seed: int, D: int, g: int, K: int, N: int) -> np.ndarray:
    """Host-side greedy pair selection -> uint8 [D/g, K, g/2, 2] (0xFF = no pair)."""
    out = np.empty((D // g, K, g // 2, 2), dtype=np.uint8)
    _check(lib.pq_select_pairs(seed, D, g, K, N, out.ctypes.data), "pq_select_pairs")
    return out


class Plan:
    """Owns a ``pq_plan`` (device tables); freed by :meth:`close` or garbage collection."""

    def __init__(self, kind, D: int, g: int = 128, K: int = 0, pairs=None, angles=None,
                 beta=None, flags: int = 0, groups8=None):
        """groups8: group indices kept as 8-bit outlier groups (codes and scales then hold
        Gx = D/g + 3 len(groups8) groups per row; see ``Dx``)."""
        kind = KINDS.get(kind, kind)
        self.kind, self.D, self.g, self.K, self.flags = kind, D, g, K, flags
        self.groups8 = [] if groups8 is None else [int(v) for v in groups8]
        self.Gx = D // g + 3 * len(self.groups8)
        self.Dx = self.Gx * g            # the GEMM's reduction length for this plan's codes
        keep = []

        def host(a, dt):
            if a is None:
                return None
            a = np.ascontiguousarray(a, dtype=dt)
            keep.append(a)
            return a.ctypes.data

        h = _vp()
        if self.groups8:
            _check(lib.pq_make_plan_outliers(_c.byref(h), kind, D, g, K, host(pairs, np.uint8),
                                             host(angles, np.float32), host(beta, np.float32), flags,
                                             len(self.groups8), host(self.groups8, np.int32)),
                   "pq_make_plan_outliers")
        else:
            _check(lib.pq_make_plan(_c.byref(h), kind, D, g, K, host(pairs, np.uint8),
                                    host(angles, np.float32), host(beta, np.float32), flags),
                   "pq_make_plan")
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib.pq_destroy_plan(self._h)
            self._h = None

    def __del__(self):  # pragma: no cover - interpreter teardown order
        try:
            self.close()
        except Exception:
            pass


def pq_make_plan(kind, D, g=128, K=0, pairs=None, angles=None, beta=None, flags=0) -> Plan:
    return Plan(kind, D, g, K, pairs, angles, beta, flags)


def pq_destroy_plan(plan: Plan) -> None:
    plan.close()


def pq_transform_quant(plan: Plan, X, codes, scales, smooth_out=None, T=None, ldx=None,
                       stream=None) -> None:
    """X bf16 [T, ldx] -> codes uint8 [T, Dx/2], scales float32 [T, Gx] (device tensors;
    Dx = D and Gx = D/g unless the plan has 8-bit groups)."""
    T = X.shape[0] if T is None else T
    ldx = X.stride(0) if ldx is None else ldx
    D, G = plan.D, plan.Gx
    if not isinstance(X, int) and X.dim() == 2 and X.stride(0) != ldx:
        raise ValueError(f"X: row stride {X.stride(0)} differs from ldx={ldx}")
    xp = _arg(X, "X", "bf16", (T - 1) * ldx + D if T > 0 else 0, rows_strided=True)
    _check(lib.pq_transform_quant(plan.handle, xp, T, ldx, _arg(codes, "codes", "u8", T * plan.Dx // 2),
                                  _arg(scales, "scales", "f32", T * G),
                                  _arg(smooth_out, "smooth_out", "f32", -(-T // 128) * D),
                                  _stream(stream)), "pq_transform_quant")


def pq_pack_weights(plan: Plan, W, codes_W, scales_W, smooth_w=None, N=None, stream=None) -> None:
    """W bf16 [N, D] -> codes_W uint8 [N, Dx/2], scales_W float32 [N, Gx] (device tensors)."""
    N = W.shape[0] if N is None else N
    D, G = plan.D, plan.Gx
    _check(lib.pq_pack_weights(plan.handle, _arg(W, "W", "bf16", N * D), N,
                               _arg(smooth_w, "smooth_w", "f32", D),
                               _arg(codes_W, "codes_W", "u8", N * plan.Dx // 2),
                               _arg(scales_W, "scales_W", "f32", N * G), _stream(stream)),
           "pq_pack_weights")


def pq_w4a4_gemm(codes_A, scales_A, codes_W, scales_W, Y, T=None, N=None, D=None, g=128,
                 out_dtype=None, stream=None) -> None:
    """Y [T, N] = per-group scaled int4 x int4 product (device tensors)."""
    T, N, D, out_dtype, ptrs = _gemm_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, g, out_dtype)
    _check(lib.pq_w4a4_gemm(*ptrs[:4], T, N, D, g, ptrs[4], out_dtype, _stream(stream)), "pq_w4a4_gemm")


def _gemm_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, g, out_dtype, sa_per_token=False):
    """Sizes, output dtype and checked pointers shared by the two GEMM entry points."""
    T = codes_A.shape[0] if T is None else T
    N = codes_W.shape[0] if N is None else N
    D = codes_A.shape[1] * 2 if D is None else D
    if not isinstance(Y, int):
        import torch
        y_kind = PQ_OUT_BF16 if Y.dtype == torch.bfloat16 else PQ_OUT_F32
        if out_dtype is None:
            out_dtype = y_kind
        elif out_dtype != y_kind or Y.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"Y: dtype {Y.dtype} does not match out_dtype={out_dtype}")
    elif out_dtype is None:
        out_dtype = PQ_OUT_F32
    G = D // g if g else 0
    ptrs = (_arg(codes_A, "codes_A", "u8", T * D // 2),
            _arg(scales_A, "token_scales" if sa_per_token else "scales_A", "f32", T if sa_per_token else T * G),
            _arg(codes_W, "codes_W", "u8", N * D // 2), _arg(scales_W, "scales_W", "f32", N * G),
            _arg(Y, "Y", "y", T * N))
    return T, N, D, out_dtype, ptrs


def pq_w4a4_gemm_noalloc(codes_A, scales_A, codes_W, scales_W, Y, T=None, N=None, D=None, g=128,
                         out_dtype=None, stream=None) -> None:
    """:func:`pq_w4a4_gemm` with the library's fixed scratch; (T + N) * D <= NOALLOC_SCRATCH_BYTES."""
    T, N, D, out_dtype, ptrs = _gemm_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, g, out_dtype)
    _check(lib.pq_w4a4_gemm_noalloc(*ptrs[:4], T, N, D, g, ptrs[4], out_dtype, _stream(stream)),
           "pq_w4a4_gemm_noalloc")


def pq_w4a4_linear(plan: Plan, X, codes_A, scales_A, codes_W, scales_W, Y, T=None, ldx=None, N=None,
                   out_dtype=None, stream=None) -> None:
    """Transform X into codes_A / scales_A and multiply with the packed weights into Y, one call
    (for T <= 128 the GEMM overlaps the transform as its programmatic dependent)."""
    T = X.shape[0] if T is None else T
    ldx = X.stride(0) if ldx is None else ldx
    N = codes_W.shape[0] if N is None else N
    D, g = plan.D, plan.g
    xp = _arg(X, "X", "bf16", (T - 1) * ldx + D if T > 0 else 0, rows_strided=True)
    T, N, _, out_dtype, ptrs = _gemm_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, plan.Dx, g, out_dtype)
    _check(lib.pq_w4a4_linear(plan.handle, xp, T, ldx, ptrs[0], ptrs[1], ptrs[2], ptrs[3], N, ptrs[4], out_dtype,
                              _stream(stream)), "pq_w4a4_linear")


def pq_rrs_prepare(plan: Plan, X, chan_max, perm, inv_perm, group_scale, T=None, ldx=None, stream=None) -> None:
    """Channel maxima of the rotated activations, their descending order and the smoothing scale
    of each reordered group of 128 (device tensors: float32 [D], int32 [D], int32 [D], float32 [G])."""
    T = X.shape[0] if T is None else T
    ldx = X.stride(0) if ldx is None else ldx
    D, G = plan.D, plan.D // plan.g
    xp = _arg(X, "X", "bf16", (T - 1) * ldx + D if T > 0 else 0, rows_strided=True)
    _check(lib.pq_rrs_prepare(plan.handle, xp, T, ldx, _arg(chan_max, "chan_max", "f32", D),
                              _arg(perm, "perm", "i32", D), _arg(inv_perm, "inv_perm", "i32", D),
                              _arg(group_scale, "group_scale", "f32", G), _stream(stream)), "pq_rrs_prepare")


def pq_rrs_transform_quant(plan: Plan, X, perm, group_scale, codes, token_scales, T=None, ldx=None,
                           stream=None) -> None:
    """Smoothed, reordered activations quantised per token: codes uint8 [T, D/2], float32 [T]."""
    T = X.shape[0] if T is None else T
    ldx = X.stride(0) if ldx is None else ldx
    D, G = plan.D, plan.D // plan.g
    xp = _arg(X, "X", "bf16", (T - 1) * ldx + D if T > 0 else 0, rows_strided=True)
    _check(lib.pq_rrs_transform_quant(plan.handle, xp, T, ldx, _arg(perm, "perm", "i32", D),
                                      _arg(group_scale, "group_scale", "f32", G),
                                      _arg(codes, "codes", "u8", T * D // 2),
                                      _arg(token_scales, "token_scales", "f32", T), _stream(stream)),
           "pq_rrs_transform_quant")


def pq_rrs_pack_weights(plan: Plan, W, perm, group_scale, codes_W, scales_W, N=None, stream=None) -> None:
    """Reordered weights quantised per group, smoothing scales folded into scales_W [N, G]."""
    N = W.shape[0] if N is None else N
    D, G = plan.D, plan.D // plan.g
    _check(lib.pq_rrs_pack_weights(plan.handle, _arg(W, "W", "bf16", N * D), N, _arg(perm, "perm", "i32", D),
                                   _arg(group_scale, "group_scale", "f32", G),
                                   _arg(codes_W, "codes_W", "u8", N * D // 2),
                                   _arg(scales_W, "scales_W", "f32", N * G), _stream(stream)),
           "pq_rrs_pack_weights")


def pq_rrs_gemm(codes_A, token_scales, codes_W, scales_W, Y, T=None, N=None, D=None, g=128, out_dtype=None,
                stream=None) -> None:
    """Y [T, N] = token_scales[t] * sum_G scales_W[n, G] d_G (device tensors)."""
    T = codes_A.shape[0] if T is None else T
    N = codes_W.shape[0] if N is None else N
    D = codes_A.shape[1] * 2 if D is None else D
    T, N, D, out_dtype, ptrs = _gemm_args(codes_A, token_scales, codes_W, scales_W, Y, T, N, D, g, out_dtype,
                                          sa_per_token=True)
    _check(lib.pq_rrs_gemm(*ptrs[:4], T, N, D, g, ptrs[4], out_dtype, _stream(stream)), "pq_rrs_gemm")


def _here():
    """Index of the current CUDA device (-1 without one) and torch, for the calls below."""
    import torch
    return (torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1), torch


def _raw_stream(stream, dev, torch):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _on(x, name, kind, dtype, need, dev):
    """:func:`_arg` and that the tensor lives on the current device (the library launches there).  is_cuda counts beside
    the device's index: without an initialised CUDA both the current device and a host tensor's are -1."""
    if x is None:
        return None
    if not isinstance(x, int) and x.dtype is dtype and x.is_cuda and x.is_contiguous() and x.numel() >= need and x.get_device() == dev:
        return x.data_ptr()
    p = _arg(x, name, kind, need)              # names what is wrong, if it is the tensor's type, layout or size
    if not isinstance(x, int) and x.get_device() != dev:
        raise ValueError(f"{name}: on {x.device}, but the current device is cuda:{dev}")
    return p


def pq_quant_rows8(X, codes, scales, g=0, T=None, D=None, ldx=None, stream=None) -> None:
    """X bf16 [T, ldx] -> codes int8 [T, D], scales float32 [T] (one a row); rows rotated in blocks of g
    channels by a Hadamard matrix first (g = 0: not)."""
    dev, torch = _here()
    xp, T, D, ldx = _rows8(X, T, D, ldx, dev, torch)
    _check(lib.pq_quant_rows8(xp, T, D, ldx, g, _on(codes, "codes", "i8", torch.int8, T * D, dev),
                              _on(scales, "scales", "f32", torch.float32, T, dev), _raw_stream(stream, dev, torch)),
           "pq_quant_rows8")


def _rows8(X, T, D, ldx, dev, torch):
    """Pointer, rows, channels and row stride of bf16 rows (a single row's stride says nothing: its length stands in).
    An ldx that is not the tensor's stride is refused: the kernels would read other rows, or past the last one."""
    if isinstance(X, int):
        return X, T, D, D if ldx is None else ldx
    if X.dim() != 2:
        raise ValueError("X: expected a 2-D tensor")
    rows, cols = X.shape
    T, D = rows if T is None else T, cols if D is None else D
    own = X.stride(0) if rows > 1 else cols
    if ldx is None:
        ldx = own
    elif ldx != own and rows > 1:
        raise ValueError(f"X: row stride {own} differs from ldx={ldx}")
    if X.dtype is not torch.bfloat16 or not X.is_cuda or X.stride(1) != 1 or T > rows or D > cols or X.get_device() != dev:
        _arg(X, "X", "bf16", (T - 1) * ldx + D if T > 0 else 0, rows_strided=True)
        if X.get_device() != dev:
            raise ValueError(f"X: on {X.device}, but the current device is cuda:{dev}")
    return X.data_ptr(), T, D, ldx


def _gemm8_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, out_dtype, dev, torch):
    if not isinstance(Y, int):
        y_kind = PQ_OUT_BF16 if Y.dtype == torch.bfloat16 else PQ_OUT_F32
        if out_dtype is None:
            out_dtype = y_kind
        elif out_dtype != y_kind:
            raise ValueError(f"Y: dtype {Y.dtype} does not match out_dtype={out_dtype}")
    elif out_dtype is None:
        out_dtype = PQ_OUT_F32
    f32, i8 = torch.float32, torch.int8
    return (out_dtype, _on(codes_A, "codes_A", "i8", i8, T * D, dev), _on(scales_A, "scales_A", "f32", f32, T, dev),
            _on(codes_W, "codes_W", "i8", i8, N * D, dev), _on(scales_W, "scales_W", "f32", f32, N, dev),
            _on(Y, "Y", "y", torch.bfloat16 if out_dtype == PQ_OUT_BF16 else f32, T * N, dev))


def pq_w8a8_gemm(codes_A, scales_A, codes_W, scales_W, Y, T=None, N=None, D=None, out_dtype=None, stream=None) -> None:
    """Y [T, N] = scales_A[t] scales_W[n] (codes_A codes_W^T), codes int8 [T, D] and [N, D]."""
    dev, torch = _here()
    T = codes_A.shape[0] if T is None else T
    N = codes_W.shape[0] if N is None else N
    D = codes_A.shape[1] if D is None else D
    out, ca, sa, cw, sw, y = _gemm8_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, out_dtype, dev, torch)
    _check(lib.pq_w8a8_gemm(ca, sa, cw, sw, T, N, D, y, out, _raw_stream(stream, dev, torch)), "pq_w8a8_gemm")


def pq_w8a8_linear(X, codes_A, scales_A, codes_W, scales_W, Y, g=0, T=None, N=None, D=None, ldx=None, out_dtype=None,
                   stream=None) -> None:
    """:func:`pq_quant_rows8` of X into codes_A / scales_A and :func:`pq_w8a8_gemm` into Y, one call."""
    dev, torch = _here()
    xp, T, D, ldx = _rows8(X, T, D, ldx, dev, torch)
    N = codes_W.shape[0] if N is None else N
    out, ca, sa, cw, sw, y = _gemm8_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, out_dtype, dev, torch)
    _check(lib.pq_w8a8_linear(xp, T, D, ldx, g, ca, sa, cw, sw, N, y, out, _raw_stream(stream, dev, torch)),
           "pq_w8a8_linear")


_call = None


class _NoModule:
    """In the compiled module's place where it is missing or does not load: no call is taken, so each is checked and made below."""
    quant_fp4 = fp4_gemm = fp4_linear = attention_masked = staticmethod(lambda *args: -1)


def _caller():
    """The compiled module behind the quickest calls (csrc/binding.cpp), loaded at the first of them: it needs torch."""
    global _call
    import importlib.machinery
    import importlib.util

    import torch                               # its libraries have to be there first

    from .build import call_lib_name
    path = os.path.join(os.path.dirname(_LIB_PATH), call_lib_name(torch.version.__version__))
    loader = importlib.machinery.ExtensionFileLoader("_pqcall", path)
    try:
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_pqcall", loader))
        module.bind(*(_c.cast(f, _vp).value for f in (lib.pq_quant_fp4, lib.pq_fp4_gemm, lib.pq_fp4_linear, lib.pq_kv4_attention_masked)))
    except ImportError as e:
        _call = _NoModule
        warnings.warn(f"calls go through ctypes, some 5 us slower: {e}; python -m rotation_int4_w4a4_b200.build makes {path}",
                      RuntimeWarning, stacklevel=3)
    else:
        _call = module
    return _call


def _fp4_format(fmt):
    form = FP4_FORMATS.get(fmt)
    if form is None:
        raise ValueError(f"fmt={fmt!r}: expected 'mx' (blocks of 32, power-of-two scales) or 'nv' (blocks of 16, E4M3 scales)")
    return form


def _fp4_group(g):
    """g as a C int holds it: the library says which are rotations."""
    if isinstance(g, int) and not -2 ** 31 <= g < 2 ** 31:
        raise ValueError(f"g={g}: expected 0, 64, 128 or 256")
    return g


def _fp4_width(codes_W, D, given):
    """Weights wider than the activations are a mistake, unless the caller has named D (narrower ones hold too little)."""
    if given is None and not isinstance(codes_W, int) and codes_W.dim() == 2 and codes_W.shape[1] * 2 > D:
        raise ValueError(f"codes_W: rows of {codes_W.shape[1]} bytes, expected {D // 2}")


def _fp4_bytes(rows, D, form):
    """Bytes of a tensor's scales (sizes the calls refuse give a small number: the library names what is wrong)."""
    span = 64 if form else 128
    return -(-rows // 128) * -(-D // span) * 512


def pq_fp4_scale_bytes(rows: int, D: int, fmt: str = "nv") -> int:
    """Size of the scale buffer (uint8) of `rows` rows of D channels."""
    n = lib.pq_fp4_scale_bytes(rows, D, _fp4_format(fmt))
    if n == 0:
        raise ValueError(f"pq_fp4_scale_bytes: {lib.pq_last_error().decode(errors='replace')}")
    return n


def pq_quant_fp4(X, codes, scales, fmt="nv", g=0, factor=1.0, T=None, D=None, ldx=None, stream=None) -> None:
    """X bf16 [T, ldx] -> E2M1 codes uint8 [T, D / 2] and one scale a block of channels, uint8 of :func:`pq_fp4_scale_bytes`
    (fmt "mx": blocks of 32, "nv": of 16, times factor); rows rotated in blocks of g channels by a Hadamard matrix first
    (g = 0: not)."""
    if T is None and D is None and ldx is None and stream is None:
        st = (_call or _caller()).quant_fp4(X, codes, scales, fmt, g, factor)
        if st >= 0:                            # -1: something is not as it should be, and is named below
            return _check(st, "pq_quant_fp4")
    dev, torch = _here()
    form = _fp4_format(fmt)
    xp, T, D, ldx = _rows8(X, T, D, ldx, dev, torch)
    u8 = torch.uint8
    _check(lib.pq_quant_fp4(xp, T, D, ldx, _fp4_group(g), form, factor, _on(codes, "codes", "u8", u8, T * D // 2, dev),
                            _on(scales, "scales", "u8", u8, _fp4_bytes(T, D, form), dev), _raw_stream(stream, dev, torch)),
           "pq_quant_fp4")


def _fp4_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, form, out_dtype, dev, torch):
    y_type = torch.bfloat16 if out_dtype == PQ_OUT_BF16 else torch.float32
    if not isinstance(Y, int):
        y_kind = PQ_OUT_BF16 if Y.dtype is torch.bfloat16 else PQ_OUT_F32
        if out_dtype is None:
            out_dtype, y_type = y_kind, torch.bfloat16 if y_kind == PQ_OUT_BF16 else torch.float32
        elif out_dtype != y_kind:
            raise ValueError(f"Y: dtype {Y.dtype} does not match out_dtype={out_dtype}")
    elif out_dtype is None:
        out_dtype = PQ_OUT_F32
    u8, half = torch.uint8, D // 2
    return (out_dtype, _on(codes_A, "codes_A", "u8", u8, T * half, dev),
            _on(scales_A, "scales_A", "u8", u8, _fp4_bytes(T, D, form), dev),
            _on(codes_W, "codes_W", "u8", u8, N * half, dev),
            _on(scales_W, "scales_W", "u8", u8, _fp4_bytes(N, D, form), dev), _on(Y, "Y", "y", y_type, T * N, dev))


def pq_fp4_gemm(codes_A, scales_A, codes_W, scales_W, Y, fmt="nv", alpha=1.0, T=None, N=None, D=None, out_dtype=None,
                stream=None) -> None:
    """Y [T, N] = alpha times the product of the numbers that E2M1 codes and their block scales stand for (codes uint8
    [T, D / 2] and [N, D / 2]; fmt "nv": alpha holds the two tensors' factors)."""
    if T is None and N is None and D is None and out_dtype is None and stream is None:
        st = (_call or _caller()).fp4_gemm(codes_A, scales_A, codes_W, scales_W, Y, fmt, alpha)
        if st >= 0:
            return _check(st, "pq_fp4_gemm")
    dev, torch = _here()
    form = _fp4_format(fmt)
    T = codes_A.shape[0] if T is None else T
    N = codes_W.shape[0] if N is None else N
    given, D = D, codes_A.shape[1] * 2 if D is None else D
    _fp4_width(codes_W, D, given)
    out, ca, sa, cw, sw, y = _fp4_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, form, out_dtype, dev, torch)
    _check(lib.pq_fp4_gemm(ca, sa, cw, sw, T, N, D, form, alpha, y, out, _raw_stream(stream, dev, torch)), "pq_fp4_gemm")


def pq_fp4_linear(X, codes_A, scales_A, codes_W, scales_W, Y, fmt="nv", g=0, factor_A=1.0, factor_W=1.0, T=None, N=None,
                  D=None, ldx=None, out_dtype=None, stream=None) -> None:
    """:func:`pq_quant_fp4` of X into codes_A / scales_A and :func:`pq_fp4_gemm` into Y, one call (fmt "nv": alpha =
    factor_A * factor_W)."""
    if T is None and N is None and D is None and ldx is None and out_dtype is None and stream is None:
        st = (_call or _caller()).fp4_linear(X, codes_A, scales_A, codes_W, scales_W, Y, fmt, g, factor_A, factor_W)
        if st >= 0:
            return _check(st, "pq_fp4_linear")
    dev, torch = _here()
    form = _fp4_format(fmt)
    given = D
    xp, T, D, ldx = _rows8(X, T, D, ldx, dev, torch)
    _fp4_width(codes_W, D, given)
    N = codes_W.shape[0] if N is None else N
    out, ca, sa, cw, sw, y = _fp4_args(codes_A, scales_A, codes_W, scales_W, Y, T, N, D, form, out_dtype, dev, torch)
    _check(lib.pq_fp4_linear(xp, T, D, ldx, _fp4_group(g), form, factor_A, ca, sa, cw, sw, factor_W, N, y, out,
                             _raw_stream(stream, dev, torch)), "pq_fp4_linear")


class KV4Cache:
    """The paged 4-bit cache of one layer: four device tensors and how they are to be read.

    k_codes, v_codes uint8 [pages, heads, page_size, head_dim / 2]; k_scales, v_scales float32 [pages, heads,
    page_size].  rotate_k / rotate_v: keys (and queries) / values are held rotated by a Hadamard matrix per head.
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales, rotate_k=True, rotate_v=True):
        shape = tuple(k_codes.shape)
        if len(shape) != 4:
            raise ValueError("k_codes: expected [pages, heads, page_size, head_dim / 2]")
        if tuple(v_codes.shape) != shape or tuple(k_scales.shape) != shape[:3] or tuple(v_scales.shape) != shape[:3]:
            raise ValueError("k_codes, v_codes, k_scales and v_scales do not have the shapes of one cache")
        if len({x.device for x in (k_codes, k_scales, v_codes, v_scales)}) != 1:
            raise ValueError("the cache's tensors are on different devices")
        n = k_scales.numel()
        self.tensors = (k_codes, k_scales, v_codes, v_scales)
        self.pages, self.heads, self.page_size, self.head_dim = shape[0], shape[1], shape[2], 2 * shape[3]
        self.rotate_k, self.rotate_v = bool(rotate_k), bool(rotate_v)
        flags = (PQ_KV4_ROTATE_K if rotate_k else 0) | (PQ_KV4_ROTATE_V if rotate_v else 0)
        self._s = _KV4Struct(_arg(k_codes, "k_codes", "u8", n * shape[3]), _arg(k_scales, "k_scales", "f32", n),
                             _arg(v_codes, "v_codes", "u8", n * shape[3]), _arg(v_scales, "v_scales", "f32", n),
                             self.pages, self.page_size, self.heads, self.head_dim, flags)
        self.handle = _c.addressof(self._s)
        self.device = k_codes.get_device()

    def on(self, dev):
        """The handle, for a call on device `dev`."""
        if dev != self.device:
            raise ValueError(f"the cache is on cuda:{self.device}, but the current device is cuda:{dev}")
        return self.handle

    @classmethod
    def empty(cls, pages, heads, page_size, head_dim, rotate_k=True, rotate_v=True, device="cuda"):
        """A cache of zeros."""
        import torch
        codes = [torch.zeros(pages, heads, page_size, head_dim // 2, dtype=torch.uint8, device=device) for _ in "kv"]
        scales = [torch.zeros(pages, heads, page_size, dtype=torch.float32, device=device) for _ in "kv"]
        return cls(codes[0], scales[0], codes[1], scales[1], rotate_k, rotate_v)


def _rows_of(x, name, width, T, dev, torch):
    """Pointer and row stride of [T, width] bf16 rows (or [T, heads, head_dim] with dense heads)."""
    shape, stride = x.shape, x.stride()
    if len(shape) == 3:
        cols = shape[1] * shape[2]
        dense = stride[2] == 1 and (stride[1] == shape[2] or shape[1] == 1)
    elif len(shape) == 2:
        cols, dense = shape[1], stride[1] == 1
    else:
        raise ValueError(f"{name}: expected [T, heads * head_dim] or [T, heads, head_dim] with dense heads")
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"{name}: dtype {x.dtype} is not accepted (expected torch.bfloat16)")
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor: the library takes device pointers")
    if not dense or cols != width or shape[0] != T:
        raise ValueError(f"{name}: shape {tuple(shape)} (strides {stride}) is not {T} rows of {width} channels")
    if x.get_device() != dev:
        raise ValueError(f"{name}: on {x.device}, but the current device is cuda:{dev}")
    return x.data_ptr(), (stride[0] if T > 1 else width)


def _query_width(Q, hd):
    w = Q.shape[1] * (Q.shape[2] if Q.dim() == 3 else 1)
    if w % hd:
        raise ValueError(f"Q: rows of {w} channels are not whole heads of {hd}")
    return w


def pq_kv4_append(cache: KV4Cache, Q, K, V, Q_out, positions, slots, rope=None, q_norm=None, k_norm=None, eps=1e-6,
                  interleaved=False, stream=None) -> None:
    """Queries, keys and values of T new tokens (bf16 rows, any row stride): norms, position rotation and Hadamard
    into Q_out bf16 [T, heads_q, head_dim] and, as 4-bit codes, into the cache at slots (int64 [T], negative: nowhere).

    rope float32 [positions, rope_dim] (cosines, then sines), positions int32 [T]; q_norm, k_norm bf16 [head_dim].
    """
    dev, torch = _here()
    T, hd = Q.shape[0], cache.head_dim
    wq, wk = _query_width(Q, hd), cache.heads * hd
    qp, ldq = _rows_of(Q, "Q", wq, T, dev, torch)
    kp, ldk = _rows_of(K, "K", wk, T, dev, torch)
    vp, ldv = _rows_of(V, "V", wk, T, dev, torch)
    rope_rows = rope_dim = 0
    if rope is not None:
        if rope.dim() != 2 or rope.numel() == 0:   # without elements it has no address: the library would see no table
            raise ValueError("rope: expected [positions, rope_dim]")
        rope_rows, rope_dim = rope.shape
    bf16 = torch.bfloat16
    _check(lib.pq_kv4_append(cache.on(dev), qp, ldq, kp, ldk, vp, ldv, T, wq // hd,
                             _on(q_norm, "q_norm", "bf16", bf16, hd, dev), _on(k_norm, "k_norm", "bf16", bf16, hd, dev), eps,
                             _on(rope, "rope", "f32", torch.float32, 0, dev), rope_rows, rope_dim,
                             _on(positions, "positions", "i32", torch.int32, T, dev),
                             _on(slots, "slots", "i64", torch.int64, T, dev), PQ_KV4_INTERLEAVED if interleaved else 0,
                             _on(Q_out, "Q_out", "bf16", bf16, T * wq, dev), _raw_stream(stream, dev, torch)),
           "pq_kv4_append")


def pq_kv4_read(cache: KV4Cache, slots, K_out, V_out, stream=None) -> None:
    """Cached rows at slots (int64 [T]) as bf16 values in the cache's basis; negative slots give zeros."""
    dev, torch = _here()
    T = slots.shape[0]
    n = T * cache.heads * cache.head_dim
    _check(lib.pq_kv4_read(cache.on(dev), _on(slots, "slots", "i64", torch.int64, T, dev), T,
                           _on(K_out, "K_out", "bf16", torch.bfloat16, n, dev),
                           _on(V_out, "V_out", "bf16", torch.bfloat16, n, dev), _raw_stream(stream, dev, torch)),
           "pq_kv4_read")


def pq_kv4_attention(cache: KV4Cache, Q, O, q_start, seq_lens, block_table, max_q, max_len, scale=None, window=0,
                     stream=None) -> None:
    """O = causal attention of the newest tokens of each sequence over its cached tokens.

    Q bf16 [T, heads_q, head_dim] as Q_out of :func:`pq_kv4_append`; q_start int32 [B + 1], seq_lens int32 [B],
    block_table int32 [B, pages of a sequence]; max_q, max_len: upper bounds (they size the launch); scale defaults
    to 1 / sqrt(head_dim); window > 0: each token sees itself and the window - 1 before it.
    """
    dev, torch = _here()
    T, hd = Q.shape[0], cache.head_dim
    wq = _query_width(Q, hd)
    qp, ldq = _rows_of(Q, "Q", wq, T, dev, torch)
    op, ldo = _rows_of(O, "O", wq, T, dev, torch)
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [sequences, pages]")
    B, width = block_table.shape
    i32 = torch.int32
    _check(lib.pq_kv4_attention(cache.on(dev), qp, ldq, wq // hd, _on(q_start, "q_start", "i32", i32, B + 1, dev),
                                _on(seq_lens, "seq_lens", "i32", i32, B, dev),
                                _on(block_table, "block_table", "i32", i32, B * width, dev), width, B, T, max_q, max_len,
                                hd ** -0.5 if scale is None else scale, window, op, ldo, _raw_stream(stream, dev, torch)),
           "pq_kv4_attention")


def pq_kv4_attention_masked(cache: KV4Cache, Q, O, q_start, seq_lens, block_table, max_q, max_len, scale=None, window=0, sinks=0,
                            tree=None, stream=None) -> None:
    """:func:`pq_kv4_attention` with sinks (under a window the first `sinks` tokens stay visible) and a tree of drafted tokens
    (int32 [T, words], 1 to 1024 words: bit j of a row's words, the lowest first, says that it sees its sequence's new token j)."""
    if stream is None:
        st = (_call or _caller()).attention_masked(cache.handle, cache.device, Q, O, q_start, seq_lens, block_table, max_q, max_len,
                                                   scale, window, sinks, tree)
        if st >= 0:
            return _check(st, "pq_kv4_attention_masked")
    dev, torch = _here()
    T, hd = Q.shape[0], cache.head_dim
    wq = _query_width(Q, hd)
    qp, ldq = _rows_of(Q, "Q", wq, T, dev, torch)
    op, ldo = _rows_of(O, "O", wq, T, dev, torch)
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [sequences, pages]")
    B, width = block_table.shape
    i32 = torch.int32
    words = 0
    if tree is not None:
        if tree.dim() != 2 or tree.shape[0] != T or tree.shape[1] < 1:   # without words it has no address: the library would see no tree
            raise ValueError(f"tree: expected [{T}, words], one word or more")
        words = tree.shape[1]
    _check(lib.pq_kv4_attention_masked(cache.on(dev), qp, ldq, wq // hd, _on(q_start, "q_start", "i32", i32, B + 1, dev),
                                       _on(seq_lens, "seq_lens", "i32", i32, B, dev),
                                       _on(block_table, "block_table", "i32", i32, B * width, dev), width, B, T, max_q,
                                       max_len, hd ** -0.5 if scale is None else scale, window, sinks,
                                       _on(tree, "tree", "i32", i32, T * words, dev), words, op, ldo,
                                       _raw_stream(stream, dev, torch)), "pq_kv4_attention_masked")


def pq_w4a4_gemm_launch_count_g(T: int, N: int, D: int, g: int) -> int:
    """Kernels one pq_w4a4_gemm call of these sizes and group size launches on the current device."""
    n = _i32(0)
    _check(lib.pq_w4a4_gemm_launch_count_g(T, N, D, g, _c.byref(n)), "pq_w4a4_gemm_launch_count_g")
    return n.value


def pq_w4a4_gemm_launch_count(T: int, N: int, D: int) -> int:
    """Kernels one pq_w4a4_gemm call of these sizes launches on the current device (2 or 3)."""
    n = _i32(0)
    _check(lib.pq_w4a4_gemm_launch_count(T, N, D, _c.byref(n)), "pq_w4a4_gemm_launch_count")
    return n.value


def pq_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch the bounded-wait diagnostic; the next pq_check_status reports PQ_ERR_TIMEOUT."""
    _check(lib.pq_selftest_wait_timeout(limit_ns, _stream(stream)), "pq_selftest_wait_timeout")


def pq_check_status(plan: Plan | None = None, stream=None) -> int:
    """Synchronise and return the status code (raises PQError on failure)."""
    st = lib.pq_check_status(plan.handle if plan is not None else None, _stream(stream))
    _check(st, "pq_check_status")
    return st
