"""Python binding of the fp4q C ABI (include/fp4q.h), through ctypes.

The functions carry the C names and do argument marshalling only: every step of the
rotate + quantize path runs in the library's CUDA kernels.  PyTorch tensors are used as
device allocations and streams.  Importing this module loads lib/libfp4q.so and raises
ImportError when it is missing; there is no fallback.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libfp4q.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"fp4q native library not built: {LIB_PATH} (run python -m "
                      "microscaling_fp4_quantization_b200.build)")

_lib = ctypes.CDLL(LIB_PATH)

FP4Q_OK, FP4Q_ERR_ARG, FP4Q_ERR_SHAPE, FP4Q_ERR_ALIGN, FP4Q_ERR_UNSUPPORTED, FP4Q_ERR_CUDA, FP4Q_ERR_TIMEOUT = range(7)
FP4Q_MXFP4, FP4Q_NVFP4, FP4Q_MXFP4_MBS = 0, 1, 2
FP4Q_KERNEL_AUTO, FP4Q_KERNEL_BUTTERFLY, FP4Q_KERNEL_TENSOR_CORE = 0, 1, 2
(FP4Q_SCALE_FLOOR_OCP, FP4Q_SCALE_CEIL_NOCLIP, FP4Q_SCALE_OAS,
 FP4Q_SCALE_NV_STATIC, FP4Q_SCALE_NV_DYNAMIC) = range(5)
FP4Q_FP8_SCALE_F32, FP4Q_FP8_SCALE_E8M0 = 0, 1
FP4Q_DTYPE_BF16, FP4Q_DTYPE_FP16, FP4Q_DTYPE_F32 = 0, 1, 2

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float

_SIGS = {
    "fp4q_plan_create": (_int, [ctypes.POINTER(_vp), _int, _int, _int, _int]),
    "fp4q_plan_destroy": (_int, [_vp]),
    "fp4q_plan_set_kernel": (_int, [_vp, _int]),
    "fp4q_plan_set_signs": (_int, [_vp, _vp, _i64]),
    "fp4q_rotate_quantize": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "fp4q_rotate_quantize_dump": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "fp4q_amax": (_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "fp4q_dequantize": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _vp]),
    "fp4q_rotate_quantize_nvfp4_dynamic_noalloc": (_int, [_vp, _i64, _i64, _int, _vp, _vp, _vp, _vp]),
    "fp4q_quant_error": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    "fp4q_rotate_quantize_mbs": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "fp4q_dequantize_mbs": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _vp]),
    "fp4q_gemm": (_int, [_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]),
    "fp4q_quantize_fp8": (_int, [_int, _int, _int, _vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "fp4q_add_rmsnorm_fp8": (_int, [_int, _int, _vp, _i64, _vp, _i64, _vp, _f32, _i64, _i64, _vp, _i64, _vp, _vp, _vp]),
    "fp4q_gemm_fp8": (_int, [_int, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]),
    "fp4q_device_status": (_int, []),
    "fp4q_selftest_wait_timeout": (_int, [_vp]),
    "fp4q_selftest_gemm_fp8_choice": (_int, [_int, _i64, _i64, _i64, _int] + [ctypes.POINTER(_int)] * 3),
    "fp4q_status_string": (ctypes.c_char_p, [_int]),
    "fp4q_last_cuda_error": (ctypes.c_char_p, []),
    "fp4q_version": (_int, []),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


class Fp4qError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.fp4q_status_string(status).decode()
        if status == FP4Q_ERR_CUDA:
            msg += ": " + _lib.fp4q_last_cuda_error().decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != FP4Q_OK:
        raise Fp4qError(status, where)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _allocating_on(stream, device):
    """A context in which torch allocates on `stream` (None: the current one), so that its allocator
    reuses a call's outputs in the order of the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    _check_stream(stream, device.index)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def _check_stream(stream, index: int) -> None:
    if not isinstance(stream, int) and stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on CUDA device {index}")


class Plan:
    """An fp4q plan handle (format, group, Hadamard block, scale rule)."""

    def __init__(self, handle: int, fmt: int, group: int, block: int, rule: int):
        self.handle = handle
        self.fmt, self.group, self.block, self.rule = fmt, group, block, rule
        self.kernel = FP4Q_KERNEL_AUTO

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            try:
                _lib.fp4q_plan_destroy(h)
            except Exception:
                pass

    @property
    def unit(self) -> int:
        return max(self.group, self.block)


# ---------------------------------------------------------------- the C names

def fp4q_plan_create(fmt: int, group: int, hadamard_block: int, scale_rule: int) -> Plan:
    h = _vp()
    _check(_lib.fp4q_plan_create(ctypes.byref(h), fmt, group, hadamard_block, scale_rule), "fp4q_plan_create")
    return Plan(h.value, fmt, group, hadamard_block, scale_rule)


def fp4q_plan_set_kernel(plan: Plan, kernel: int) -> None:
    _check(_lib.fp4q_plan_set_kernel(plan.handle, kernel), "fp4q_plan_set_kernel")
    plan.kernel = kernel


def fp4q_plan_set_signs(plan: Plan, signs, K: int) -> None:
    """signs: device uint32 tensor [ceil(K/32)] (bit k negates channel k) or None to clear.
    The plan keeps a reference to the tensor so that it stays alive."""
    _check(_lib.fp4q_plan_set_signs(plan.handle, _ptr(signs), K), "fp4q_plan_set_signs")
    plan.signs = signs


def fp4q_plan_destroy(plan: Plan) -> None:
    h, plan.handle = plan.handle, None
    _check(_lib.fp4q_plan_destroy(h), "fp4q_plan_destroy")


def fp4q_rotate_quantize(plan: Plan, x, M: int, K: int, codes_out, scales_out, tensor_scale=None,
                         stream=None) -> None:
    _check(_lib.fp4q_rotate_quantize(plan.handle, _ptr(x), M, K, _ptr(codes_out), _ptr(scales_out),
                                     _ptr(tensor_scale), _stream(stream)), "fp4q_rotate_quantize")


def fp4q_rotate_quantize_dump(plan: Plan, x, M: int, K: int, codes_out, scales_out, tensor_scale, y_out,
                              stream=None) -> None:
    _check(_lib.fp4q_rotate_quantize_dump(plan.handle, _ptr(x), M, K, _ptr(codes_out), _ptr(scales_out),
                                          _ptr(tensor_scale), _ptr(y_out), _stream(stream)),
           "fp4q_rotate_quantize_dump")


def fp4q_amax(plan: Plan, x, M: int, K: int, tensor_scale_out, stream=None) -> None:
    _check(_lib.fp4q_amax(plan.handle, _ptr(x), M, K, _ptr(tensor_scale_out), _stream(stream)), "fp4q_amax")


def fp4q_dequantize(plan: Plan, codes, scales, tensor_scale, M: int, K: int, unrotate: bool, out_f32,
                    stream=None) -> None:
    _check(_lib.fp4q_dequantize(plan.handle, _ptr(codes), _ptr(scales), _ptr(tensor_scale), M, K,
                                int(bool(unrotate)), _ptr(out_f32), _stream(stream)), "fp4q_dequantize")


def fp4q_rotate_quantize_nvfp4_dynamic_noalloc(x, M: int, K: int, hadamard_block: int, codes_out, scales_out,
                                                tensor_scale_out, stream=None) -> None:
    """NVFP4 dynamic-scale rotate + quantize without any device allocation (its scratch is a
    fixed array inside the library); for callers that cannot allocate device memory."""
    _check(_lib.fp4q_rotate_quantize_nvfp4_dynamic_noalloc(_ptr(x), M, K, hadamard_block, _ptr(codes_out),
                                                           _ptr(scales_out), _ptr(tensor_scale_out),
                                                           _stream(stream)),
           "fp4q_rotate_quantize_nvfp4_dynamic_noalloc")


def fp4q_quant_error(plan: Plan, x, M: int, K: int, tensor_scale, out_f64, stream=None) -> None:
    """out_f64: device float64 [3] <- {signal energy, error energy, QSNR dB}."""
    _check(_lib.fp4q_quant_error(plan.handle, _ptr(x), M, K, _ptr(tensor_scale), _ptr(out_f64), _stream(stream)),
           "fp4q_quant_error")


def fp4q_rotate_quantize_mbs(plan: Plan, x, M: int, K: int, codes_out, scales_out, macro_out, stream=None) -> None:
    _check(_lib.fp4q_rotate_quantize_mbs(plan.handle, _ptr(x), M, K, _ptr(codes_out), _ptr(scales_out),
                                         _ptr(macro_out), _stream(stream)), "fp4q_rotate_quantize_mbs")


def fp4q_dequantize_mbs(plan: Plan, codes, scales, macro, M: int, K: int, unrotate: bool, out_f32,
                        stream=None) -> None:
    _check(_lib.fp4q_dequantize_mbs(plan.handle, _ptr(codes), _ptr(scales), _ptr(macro), M, K, int(bool(unrotate)),
                                    _ptr(out_f32), _stream(stream)), "fp4q_dequantize_mbs")


def fp4q_gemm(fmt: int, a_codes, a_scales, a_tensor_scale, b_codes, b_scales, b_tensor_scale, M: int, N: int,
              K: int, d_bf16, stream=None) -> None:
    """D [M, N] bf16 = alpha * A B^T from the quantizer's codes and scales of A [M, K] and B [N, K]."""
    _check(_lib.fp4q_gemm(fmt, _ptr(a_codes), _ptr(a_scales), _ptr(a_tensor_scale), _ptr(b_codes), _ptr(b_scales),
                          _ptr(b_tensor_scale), M, N, K, _ptr(d_bf16), _stream(stream)), "fp4q_gemm")


def fp4q_quantize_fp8(scale_format: int, dtype: int, block_rows: int, x, ldx: int, M: int, K: int, codes_out,
                      scales_out, stream=None) -> None:
    """E4M3 codes [M, K] and scales of x (rows ldx elements apart): block_rows 1 for a scale per row and
    128 channels, 128 for a scale per 128 x 128 tile."""
    _check(_lib.fp4q_quantize_fp8(scale_format, dtype, block_rows, _ptr(x), ldx, M, K, _ptr(codes_out),
                                  _ptr(scales_out), _stream(stream)), "fp4q_quantize_fp8")


def fp4q_add_rmsnorm_fp8(scale_format: int, dtype: int, x, ldx: int, residual, ldr: int, weight, eps: float, M: int,
                         K: int, residual_out, ldo: int, codes_out, scales_out, stream=None) -> None:
    """residual_out = x + residual, and E4M3 codes and scales (per row and 128 channels) of its RMS norm."""
    _check(_lib.fp4q_add_rmsnorm_fp8(scale_format, dtype, _ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), eps, M, K,
                                     _ptr(residual_out), ldo, _ptr(codes_out), _ptr(scales_out), _stream(stream)),
           "fp4q_add_rmsnorm_fp8")


def fp4q_gemm_fp8(scale_format: int, out_dtype: int, a_codes, a_scales, b_codes, b_scales, M: int, N: int, K: int, d,
                  stream=None) -> None:
    """D [M, N] = A B^T from the codes and scales of A [M, K] (block_rows 1) and B [N, K] (block_rows 128)."""
    _check(_lib.fp4q_gemm_fp8(scale_format, out_dtype, _ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales),
                              M, N, K, _ptr(d), _stream(stream)), "fp4q_gemm_fp8")


def fp4q_device_status() -> int:
    return _lib.fp4q_device_status()


def fp4q_selftest_wait_timeout(stream=None) -> None:
    """One warp whose bounded wait runs out: the next fp4q_device_status is FP4Q_ERR_TIMEOUT."""
    _check(_lib.fp4q_selftest_wait_timeout(_stream(stream)), "fp4q_selftest_wait_timeout")


def fp4q_selftest_gemm_fp8_choice(scale_format: int, M: int, N: int, K: int, sm_count: int = 0) -> Tuple[int, int, int]:
    """(rows, columns) of the tile of D that fp4q_gemm_fp8 takes for these sizes, and the CTAs K is split over."""
    out = [_int() for _ in range(3)]
    _check(_lib.fp4q_selftest_gemm_fp8_choice(scale_format, M, N, K, sm_count, *map(ctypes.byref, out)),
           "fp4q_selftest_gemm_fp8_choice")
    return tuple(v.value for v in out)


def fp4q_status_string(status: int) -> str:
    return _lib.fp4q_status_string(status).decode()


def fp4q_version() -> int:
    return _lib.fp4q_version()


def raw_call(name: str, *args) -> int:
    """Call a C entry point with raw arguments and return its status (for tests of the
    host-side argument checks)."""
    return getattr(_lib, name)(*args)


# ---------------------------------------------------------------- tensor conveniences
#
# `stream`: a torch.cuda.Stream or a stream's handle; None is the current stream.  A call's outputs are
# allocated on the stream it runs on.  An input that lives on another stream is the caller's to order
# before the call, and to keep (or to record with Tensor.record_stream) until the call's stream has read it.

def empty_outputs(plan: Plan, M: int, K: int, device="cuda"):
    """Allocate codes (uint8 [M, K/2]), scales (uint8 [M, K/g]) and the fp32 tensor scale."""
    import torch
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((M, K // plan.group), dtype=torch.uint8, device=device)
    ts = torch.empty((1,), dtype=torch.float32, device=device)
    return codes, scales, ts


def rotate_quantize(plan: Plan, x, tensor_scale=None, stream=None) -> Tuple[object, object, object]:
    """x: bf16 CUDA tensor [M, K] -> (codes, scales, tensor_scale)."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bf16 CUDA tensor")
    M, K = x.shape
    with _allocating_on(stream, x.device):
        codes, scales, ts = empty_outputs(plan, M, K, x.device)
    if tensor_scale is not None:
        ts = tensor_scale
    fp4q_rotate_quantize(plan, x, M, K, codes, scales, ts if plan.fmt == FP4Q_NVFP4 else None, stream)
    return codes, scales, ts


def quant_error(plan: Plan, x, tensor_scale=None, stream=None):
    """x: bf16 CUDA tensor [M, K] -> (signal, error, qsnr_db) as Python floats (synchronises)."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bf16 CUDA tensor")
    M, K = x.shape
    with _allocating_on(stream, x.device):   # the read back waits for that stream too
        out = torch.empty(3, dtype=torch.float64, device=x.device)
        ts = tensor_scale
        if plan.fmt == FP4Q_NVFP4 and ts is None:
            ts = torch.empty(1, dtype=torch.float32, device=x.device)
        fp4q_quant_error(plan, x, M, K, ts, out, stream)
        s, e, q = out.tolist()
    return s, e, q


# ---- 8-bit linear layers.  Codes are torch.float8_e4m3fn tensors, scales float32 or torch.float8_e8m0fnu
# ones.  The calls run on the tensors' device, on its current stream unless one is given.  The checks are
# written for few attribute reads: at one token a call costs the host more than it costs the GPU.

_torch = None            # set by the first call: importing this module does not import torch
_e4m3 = None
_raw_stream = None       # device index -> handle of its current stream (current_stream() takes 3 us to say it)
_current_device = None
_fp8_in_dtypes: dict = {}      # input types, and their codes
_fp8_out_dtypes: dict = {}
_fp8_scale_dtypes: dict = {}


def _fp8_init() -> None:
    global _torch, _e4m3, _raw_stream, _current_device
    import torch
    _fp8_in_dtypes.update({torch.bfloat16: FP4Q_DTYPE_BF16, torch.float16: FP4Q_DTYPE_FP16})
    _fp8_out_dtypes.update(_fp8_in_dtypes)
    _fp8_out_dtypes[torch.float32] = FP4Q_DTYPE_F32
    _fp8_scale_dtypes[FP4Q_FP8_SCALE_F32] = torch.float32
    if hasattr(torch, "float8_e8m0fnu"):   # else only float32 scales are offered
        _fp8_scale_dtypes[FP4Q_FP8_SCALE_E8M0] = torch.float8_e8m0fnu
    _e4m3 = torch.float8_e4m3fn
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # (not a public name)
    if _raw_stream is None:
        _raw_stream = lambda index: torch.cuda.current_stream(index).cuda_stream
    _current_device = torch.cuda.current_device
    _torch = torch


def _fp8_ld(name: str, t) -> int:
    """The distance between the rows of a 2-D tensor whose rows are contiguous."""
    M, K = t.shape
    if K > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if M > 1 and K > 0 else K


def _fp8_like(name: str, t, shape, dtype, index) -> int:
    """Check a tensor that goes with x; returns the distance between its rows."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must match x in shape, dtype and device")
    return shape[1] if t.is_contiguous() else _fp8_ld(name, t)


def _fp8_array(name: str, t, shape, dtype, index):
    """Check a contiguous tensor."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device {index}")
    return t


def _fp8_empty(shape, dtype, index, stream):
    """An output of a call on `stream`."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=index)
    with _allocating_on(stream, _torch.device("cuda", index)):
        return _torch.empty(shape, dtype=dtype, device=index)


def _fp8_call(name: str, index: int, stream, *args) -> None:
    """The C call `name` on the device's current stream, or on the given one, with the device current."""
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        _check_stream(stream, index)
        stream = stream.cuda_stream
    if _current_device() == index:
        status = getattr(_lib, name)(*args, stream)
    else:
        with _torch.cuda.device(index):
            status = getattr(_lib, name)(*args, stream)
    if status:
        raise Fp4qError(status, name)


def quantize_fp8(x, block_rows: int = 1, scale_format: int = FP4Q_FP8_SCALE_F32, codes=None, scales=None, stream=None):
    """x: bf16 or fp16 CUDA tensor [M, K] (K a multiple of 16; rows may be strided) -> (codes
    float8_e4m3fn [M, K], scales).  block_rows 1: scales [M, ceil(K / 128)], for activations; 128:
    [ceil(M / 128), ceil(K / 128)], for weights.  scale_format: FP4Q_FP8_SCALE_F32 (float32 scales) or
    FP4Q_FP8_SCALE_E8M0 (float8_e8m0fnu).  codes, scales: outputs to write into."""
    if _torch is None:
        _fp8_init()
    shape, dtype, index = x.shape, _fp8_in_dtypes.get(x.dtype), x.get_device()
    if dtype is None or index < 0 or len(shape) != 2:
        raise ValueError("x must be a 2-D bf16 or fp16 CUDA tensor")
    s_dtype = _fp8_scale_dtypes.get(scale_format)
    if s_dtype is None or block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128 and scale_format one of FP4Q_FP8_SCALE_*")
    M, K = shape
    ldx = K if x.is_contiguous() else _fp8_ld("x", x)
    s_shape = (-(-M // block_rows), -(-K // 128))
    codes = _fp8_empty(shape, _e4m3, index, stream) if codes is None else \
        _fp8_array("codes", codes, shape, _e4m3, index)
    scales = _fp8_empty(s_shape, s_dtype, index, stream) if scales is None else \
        _fp8_array("scales", scales, s_shape, s_dtype, index)
    _fp8_call("fp4q_quantize_fp8", index, stream, scale_format, dtype, block_rows, x.data_ptr(), ldx, M, K,
              codes.data_ptr(), scales.data_ptr())
    return codes, scales


def add_rmsnorm_fp8(x, residual, weight, eps: float, scale_format: int = FP4Q_FP8_SCALE_F32, residual_out=None,
                    codes=None, scales=None, stream=None):
    """h = x + residual (residual None: x alone), y = h / sqrt(mean(h^2) + eps) * weight -> (codes
    float8_e4m3fn [M, K] and scales [M, ceil(K / 128)] of y, residual_out = h in x's dtype or None).
    x, residual [M, K] and weight [K]: bf16 or fp16, of one dtype; rows may be strided.  residual_out may
    be given: residual or x itself, or another tensor that overlaps neither."""
    if _torch is None:
        _fp8_init()
    shape, t_dtype, index = x.shape, x.dtype, x.get_device()
    dtype, s_dtype = _fp8_in_dtypes.get(t_dtype), _fp8_scale_dtypes.get(scale_format)
    if dtype is None or index < 0 or len(shape) != 2:
        raise ValueError("x must be a 2-D bf16 or fp16 CUDA tensor")
    if s_dtype is None:
        raise ValueError("scale_format must be one of FP4Q_FP8_SCALE_*")
    M, K = shape
    ldx = K if x.is_contiguous() else _fp8_ld("x", x)
    _fp8_array("weight", weight, (K,), t_dtype, index)
    ldr = ldo = K
    p_res = p_out = None
    if residual is not None:
        ldr = _fp8_like("residual", residual, shape, t_dtype, index)
        if residual_out is None:
            residual_out = _fp8_empty(shape, t_dtype, index, stream)
        else:
            ldo = _fp8_like("residual_out", residual_out, shape, t_dtype, index)
        p_res, p_out = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out goes with a residual")
    s_shape = (M, -(-K // 128))
    codes = _fp8_empty(shape, _e4m3, index, stream) if codes is None else \
        _fp8_array("codes", codes, shape, _e4m3, index)
    scales = _fp8_empty(s_shape, s_dtype, index, stream) if scales is None else \
        _fp8_array("scales", scales, s_shape, s_dtype, index)
    if M > 0 and K > 0:   # (an empty tensor's null pointers say nothing about a residual)
        _fp8_call("fp4q_add_rmsnorm_fp8", index, stream, scale_format, dtype, x.data_ptr(), ldx, p_res, ldr,
                  weight.data_ptr(), eps, M, K, p_out, ldo, codes.data_ptr(), scales.data_ptr())
    return codes, scales, residual_out


def gemm_fp8(a_codes, a_scales, b_codes, b_scales, out_dtype=None, out=None, stream=None):
    """D = A B^T [M, N] from A's codes [M, K] and scales [M, ceil(K / 128)] (quantize_fp8 or
    add_rmsnorm_fp8) and B's codes [N, K] and scales [ceil(N / 128), ceil(K / 128)] (quantize_fp8 with
    block_rows 128); both scales float32 or both float8_e8m0fnu.  out_dtype: bf16 (the default), fp16 or
    fp32.  out: a tensor to write into."""
    if _torch is None:
        _fp8_init()
    shape, b_shape, s_dtype, index = a_codes.shape, b_codes.shape, a_scales.dtype, a_codes.get_device()
    if len(shape) != 2 or len(b_shape) != 2 or index < 0:
        raise ValueError("a_codes [M, K] and b_codes [N, K] must be 2-D CUDA tensors")
    (M, K), N = shape, b_shape[0]
    kb = -(-K // 128)
    fmt = FP4Q_FP8_SCALE_F32 if s_dtype is _torch.float32 else FP4Q_FP8_SCALE_E8M0
    if s_dtype is not _fp8_scale_dtypes.get(fmt):
        raise ValueError("the scales must be float32 or float8_e8m0fnu")
    _fp8_array("a_codes", a_codes, shape, _e4m3, index)
    _fp8_array("b_codes", b_codes, (N, K), _e4m3, index)
    _fp8_array("a_scales", a_scales, (M, kb), s_dtype, index)
    _fp8_array("b_scales", b_scales, (-(-N // 128), kb), s_dtype, index)
    if out_dtype is None:
        out_dtype = _torch.bfloat16 if out is None else out.dtype
    dtype = _fp8_out_dtypes.get(out_dtype)
    if dtype is None:
        raise ValueError("out_dtype must be bf16, fp16 or fp32")
    out = _fp8_empty((M, N), out_dtype, index, stream) if out is None else \
        _fp8_array("out", out, (M, N), out_dtype, index)
    _fp8_call("fp4q_gemm_fp8", index, stream, fmt, dtype, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(),
              b_scales.data_ptr(), M, N, K, out.data_ptr())
    return out
