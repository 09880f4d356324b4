"""Python binding of libgemma_nq.so: argument marshalling only.

Every step of the operation runs in the library's CUDA kernels; this module
checks tensor metadata, allocates outputs with PyTorch the way
"vllm.models.qwen3_5.nvidia.ops.fused_norm_quant" (gemma_add_rms_norm_quant)
does, passes raw pointers (CUDA or pinned host memory) and the current CUDA
stream through ctypes,
and turns a nonzero status into an exception.  There is no fallback: if the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

GNQ_OK = 0
_DTYPE = {torch.bfloat16: 0, torch.float16: 1}
_MODES = {"none": -1, "fp8": 0, "nvfp4": 1, "mxfp8": 2}

_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load the in-tree libgemma_nq.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        P, i64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        sigs = {
            "gemma_add_rms_norm": [P, P, P, F, P, i64, i64, I, P],
            "gemma_add_rms_norm_quant": [P, P, P, F, P, I, I, P, P, P, i64, i64, I, P],
            "gemma_add_rms_norm_quant_parts": [P, I, i64, P, P, F, P, I, I, P, P, P, i64, i64, I, P],
            "add_rms_norm_quant": [P, I, i64, P, P, F, P, I, I, P, P, P, i64, i64, I, P],
            "gemma_sandwich_norm_quant": [P, P, P, P, P, P, i64, F, F, P, I, I, P, P, P, i64, i64, I, P],
            "gnq_quantize": [P, i64, P, I, P, P, i64, i64, I, P],
            "gated_act_quant": [P, i64, I, P, I, I, P, P, P, i64, i64, I, P],
            "gnq_nvfp4_dequantize": [P, P, P, P, i64, i64, I, P],
            "nvfp4_linear": [P, P, P, P, P, P, P, i64, i64, i64, I, I, P],
            "gnq_set_launch_policy": [I, I, I, I],
            "gnq_set_linear_policy": [I],
            "gnq_query_linear": [i64, i64, i64, I, P, P, P],
            "gnq_query_launch": [i64, i64, I, I, I, I, I, F, P, P, P, P],
            "gnq_read_device_error": [P, I],
            "gnq_set_pdl": [I],
            "gnq_set_constant_weights": [I],
            "gnq_inject_wait_timeout": [I],
            "gnq_inject_split_timeout": [I],
            "gnq_quantize_fp8_values": [P, i64, P, P, P],
            "gnq_pdl_consumer": [P, i64, P, i64, P, I, P],
            "gnq_encode_e4m3_e2m1": [P, i64, P, P, P],
        }
        for name, argt in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes = argt
            fn.restype = ctypes.c_int
        lib.gnq_status_string.argtypes = [ctypes.c_int]
        lib.gnq_status_string.restype = ctypes.c_char_p
        _lib = lib
        return lib


# Names the C ABI exports (checked by the test suite against include/gemma_nq.h).
EXPORTS = ("gemma_add_rms_norm", "gemma_add_rms_norm_quant", "gemma_add_rms_norm_quant_parts",
           "add_rms_norm_quant", "gnq_status_string", "gnq_set_launch_policy",
           "gnq_read_device_error", "gnq_set_pdl", "gnq_encode_e4m3_e2m1",
           "gnq_quantize_fp8_values", "gnq_query_launch", "gnq_set_constant_weights",
           "gnq_inject_wait_timeout", "gnq_inject_split_timeout", "gnq_pdl_consumer", "gemma_sandwich_norm_quant",
           "gnq_set_linear_policy", "gnq_query_linear", "gnq_quantize", "gated_act_quant", "gnq_nvfp4_dequantize", "nvfp4_linear")


def status_string(status: int) -> str:
    return load().gnq_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != GNQ_OK:
        raise RuntimeError(f"{what}: {status_string(status)} (status {status})")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _mode(mode) -> int:
    if isinstance(mode, bool):  # the pages' signature: nvfp4=True / False
        return _MODES["nvfp4"] if mode else _MODES["fp8"]
    if isinstance(mode, str):
        return _MODES[mode]
    return int(mode)


def _reachable(t: torch.Tensor) -> bool:
    """A tensor the GPU can address: CUDA memory or pinned (mapped) host memory."""
    return t.is_cuda or t.is_pinned()


def _check_act(x: torch.Tensor, name: str) -> None:
    if not _reachable(x) or not x.is_contiguous() or x.dtype not in _DTYPE:
        raise ValueError(f"{name} must be a contiguous bf16/fp16 tensor in CUDA or pinned memory")


def _check_buf(t, name: str, nbytes: int, dtype=None, required: bool = True) -> None:
    """A buffer the kernels read or write: contiguous, of `dtype` if given, at
    least `nbytes` long, in CUDA or pinned memory.  Raises before any launch
    (the library itself cannot see a buffer's size)."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required here")
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes; the call needs {nbytes}")
    if not _reachable(t):
        raise ValueError(f"{name} must be in CUDA or pinned host memory")


def _check_call(M: int, H: int, k: int, dt, residual, weight, mode: int, write_y: bool, out):
    """Sizes of every buffer a call touches (x itself checked by the caller)."""
    e = 2
    _check_buf(residual, "residual", M * H * e, dt, required=False)
    _check_buf(weight, "weight", H * e, dt)
    q, bs, y = out
    if mode in (0, 2):
        _check_buf(q, "q", M * H)
    elif mode == 1:
        _check_buf(q, "q", M * H // 2)
    if mode == 1:
        _check_buf(bs, "block_scale", round_up(M, 128) * round_up(H // 16, 4))
    elif mode == 2:
        _check_buf(bs, "block_scale", M * (H // 32))
    if write_y or mode == -1:
        _check_buf(y, "y", M * H * e, dt)


def round_up(a: int, b: int) -> int:
    return (a + b - 1) // b * b


def alloc_outputs(M: int, H: int, mode, write_y: bool, like: torch.Tensor):
    """(q, block_scale, y) buffers as the pages allocate them; block_scale is
    None for FP8 (whose block scale is the static scale tensor).  Placed like
    `like`: on its CUDA device, or in pinned host memory for a host tensor."""
    m = _mode(mode)
    kw = {"device": like.device} if like.is_cuda else {"pin_memory": True}
    q = bs = None
    if m in (0, 2):
        q = torch.empty((M, H), dtype=torch.float8_e4m3fn, **kw)
    elif m == 1:
        q = torch.empty((M, H // 2), dtype=torch.uint8, **kw)
    if m == 1:
        bs = torch.empty((round_up(M, 128), round_up(H // 16, 4) // 4), dtype=torch.int32,
                         **kw).view(torch.float8_e4m3fn)
    elif m == 2:
        bs = torch.empty((M, H // 32), dtype=torch.uint8, **kw)
    y = torch.empty((M, H), dtype=like.dtype, **kw) if (write_y or m == -1) else None
    return q, bs, y


def gemma_add_rms_norm(x, residual, weight, eps, y=None, stream=None):
    """Residual add + Gemma RMSNorm.  Returns (y, residual); residual (if
    given) is updated in place to x + residual."""
    _check_act(x, "x")
    M, H = x.shape
    if y is None:
        y = torch.empty_like(x) if x.is_cuda else torch.empty(x.shape, dtype=x.dtype, pin_memory=True)
    _check_call(M, H, 1, x.dtype, residual, weight, -1, True, (None, None, y))
    st = load().gemma_add_rms_norm(_ptr(x), _ptr(residual), _ptr(weight), float(eps), _ptr(y),
                                   M, H, _DTYPE[x.dtype], _stream(stream))
    _check(st, "gemma_add_rms_norm")
    return y, residual


def _scale_ptr(scale):
    if scale is None:
        return None
    if not (_reachable(scale) and scale.dtype == torch.float32 and scale.numel() == 1):
        raise ValueError("scale must be a 1-element fp32 tensor in CUDA or pinned memory")
    return _ptr(scale)


def gemma_add_rms_norm_quant(x, residual, weight, eps, scale, nvfp4=False, write_y=False,
                             out=None, stream=None):
    """Gemma RMSNorm of x (+ residual) quantized for the next linear.

    ``nvfp4`` may be a bool (the pages' signature) or one of "fp8", "nvfp4",
    "mxfp8".  Returns (q, block_scale, y) like the pages' op: block_scale is
    the swizzled E4M3 scale tensor for NVFP4, the (M, H/32) E8M0 codes for
    MXFP8, and ``scale`` itself for FP8; y is None unless write_y.  ``out``
    may supply preallocated (q, block_scale, y)."""
    _check_act(x, "x")
    M, H = x.shape
    m = _mode(nvfp4)
    q, bs, y = out if out is not None else alloc_outputs(M, H, m, write_y, x)
    _check_call(M, H, 1, x.dtype, residual, weight, m, write_y, (q, bs, y))
    st = load().gemma_add_rms_norm_quant(
        _ptr(x), _ptr(residual), _ptr(weight), float(eps), _scale_ptr(scale), m,
        1 if write_y else 0, _ptr(q), _ptr(bs), _ptr(y), M, H, _DTYPE[x.dtype], _stream(stream))
    _check(st, "gemma_add_rms_norm_quant")
    return q, (scale if m == 0 else bs), (y if write_y else None)


def _parts_call(fn_name, x_parts, residual, weight, eps, scale, mode, write_y, out, stream):
    if x_parts.dim() == 2:
        x_parts = x_parts.unsqueeze(0)
    if not _reachable(x_parts) or not x_parts.is_contiguous() or x_parts.dtype not in _DTYPE:
        raise ValueError("x_parts must be a contiguous bf16/fp16 tensor (k, M, H) in CUDA or "
                         "pinned memory")
    k, M, H = x_parts.shape
    m = _mode(mode)
    q, bs, y = out if out is not None else alloc_outputs(M, H, m, write_y, x_parts)
    _check_call(M, H, k, x_parts.dtype, residual, weight, m, write_y, (q, bs, y))
    st = getattr(load(), fn_name)(
        _ptr(x_parts), k, M * H, _ptr(residual), _ptr(weight), float(eps), _scale_ptr(scale), m,
        1 if (write_y or m == -1) else 0, _ptr(q), _ptr(bs), _ptr(y), M, H,
        _DTYPE[x_parts.dtype], _stream(stream))
    _check(st, fn_name)
    return q, (scale if m == 0 else bs), (y if (write_y or m == -1) else None)


def gemma_add_rms_norm_quant_parts(x_parts, residual, weight, eps, scale, mode, write_y=False,
                                   out=None, stream=None):
    """As gemma_add_rms_norm_quant with the activation given as k partial
    buffers (k, M, H), summed in fp32 on the GPU before the residual add."""
    return _parts_call("gemma_add_rms_norm_quant_parts", x_parts, residual, weight, eps, scale,
                       mode, write_y, out, stream)


def add_rms_norm_quant(x_parts, residual, weight, eps, scale, mode, write_y=False, out=None,
                       stream=None):
    """Plain RMSNorm variant (y = h * rsqrt(mean(h^2) + eps) * w)."""
    return _parts_call("add_rms_norm_quant", x_parts, residual, weight, eps, scale, mode,
                       write_y, out, stream)


_OUT_TYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
_ACTS = {"silu": 1, "gelu_tanh": 2}


def _need(t, name: str, nbytes: int, dtypes, contiguous: bool = True) -> None:
    """A buffer of one of `dtypes`, at least `nbytes` long."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a tensor of {' / '.join(str(d) for d in dtypes)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes; the call needs {nbytes}")


def _place(tensors, pinned: bool = True) -> int:
    """The device of a call: every tensor on the current CUDA device (or, where
    the operator takes it, in pinned host memory)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if t.is_cuda:
            if dev is None:
                dev = torch.cuda.current_device()
            if t.get_device() != dev:
                raise ValueError(f"a tensor is on cuda:{t.get_device()}, but the current device is cuda:{dev}")
        elif not pinned or not t.is_pinned():
            raise ValueError("tensors must be in CUDA" + (" or pinned host memory" if pinned else " memory"))
    return torch.cuda.current_device() if dev is None else dev


def _rows(x, name: str):
    """(rows, columns, row stride) of a 2-D 16-bit matrix with dense rows."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in _DTYPE:
        raise ValueError(f"{name} must be a 2-D bf16/fp16 tensor")
    M, W = x.shape
    sm, sn = x.stride()
    if W > 1 and sn != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return M, W, (sm if M > 1 else W)


def _need_outputs(M: int, H: int, m: int, dt, write_y: bool, out) -> None:
    q, bs, y = out
    if m in (0, 2):
        _need(q, "q", M * H, (torch.float8_e4m3fn, torch.uint8))
    elif m == 1:
        _need(q, "q", M * H // 2, (torch.uint8,))
        _need(bs, "block_scale", round_up(M, 128) * (H // 16), (torch.float8_e4m3fn, torch.uint8))
    if m == 2:
        _need(bs, "block_scale", M * (H // 32), (torch.uint8,))
    if write_y:
        _need(y, "y", M * H * 2, (dt,))


def _need_scale(scale, name: str, required: bool) -> None:
    if scale is None and not required:
        return
    if not isinstance(scale, torch.Tensor) or scale.dtype != torch.float32 or scale.numel() != 1:
        raise ValueError(f"{name} must be a 1-element fp32 tensor")


# Each call below first tries its whole argument check as one expression (all
# tensors on the current CUDA device, the common case: a call of a decode step
# takes microseconds, most of them here); what that does not pass goes through
# the step-by-step check, which names the fault or admits pinned host memory.
_U8, _F32, _E4M3 = torch.uint8, torch.float32, torch.float8_e4m3fn
# the current device and its current stream, without torch.cuda's wrappers
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _outputs_ok(dev: int, M: int, H: int, m: int, dt, write_y: bool, q, bs, y) -> bool:
    if write_y and not (y.dtype is dt and y.is_contiguous() and y.nbytes >= 2 * M * H and y.get_device() == dev):
        return False
    if m == 1:
        return (q.dtype is _U8 and q.is_contiguous() and q.nbytes >= M * H // 2 and q.get_device() == dev
                and bs.dtype in (_E4M3, _U8) and bs.is_contiguous()
                and bs.nbytes >= (M + 127) // 128 * 8 * H and bs.get_device() == dev)
    if m == -1:
        return True
    return (q.dtype in (_E4M3, _U8) and q.is_contiguous() and q.nbytes >= M * H and q.get_device() == dev
            and (m == 0 or (bs.dtype is _U8 and bs.is_contiguous() and bs.nbytes >= M * (H // 32)
                            and bs.get_device() == dev)))


def _scale_ok(dev: int, m: int, scale) -> bool:
    if scale is None:
        return m in (-1, 2)
    return scale.dtype is _F32 and scale.numel() == 1 and scale.get_device() == dev


def _gate_stride(gate, M: int, H: int, dt) -> int:
    if isinstance(gate, torch.Tensor) and gate.dtype == dt:
        if gate.dim() == 2 and gate.shape == (M, H):
            return _rows(gate, "gate")[2]
        if gate.shape == (H,) and gate.is_contiguous():
            return 0
    raise ValueError(f"gate must be a ({H},) or ({M}, {H}) tensor of {dt}")


def gemma_sandwich_norm_quant(x, residual, post_weight, weight, eps, scale=None, mode="nvfp4", gate=None,
                              residual_scale=1.0, residual_out=None, write_y=False, out=None, stream=None):
    """The norm after a block, its gate and residual scale, the residual add,
    and the norm before the next block quantized for its first linear:

        u = x * rsqrt(mean(x^2) + eps) * (1 + post_weight)   (u = x without one)
        h = residual + residual_scale * gate * u             (rounded once)
        q = quant(y), y = h * rsqrt(mean(h^2) + eps) * (1 + weight)

    ``gate`` is None, (H,) or (M, H) with dense rows.  h goes to
    ``residual_out``, or in place to ``residual``.  ``mode`` is "none" (y
    only), "fp8", "nvfp4" or "mxfp8"; ``out`` may supply (q, block_scale, y).
    Returns (q, block_scale, y) as gemma_add_rms_norm_quant does."""
    m = _MODES[mode] if type(mode) is str else _mode(mode)
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in _DTYPE:
        raise ValueError("x must be a 2-D bf16/fp16 tensor")
    M, H = x.shape
    dt = x.dtype
    write_y = bool(write_y) or m == -1
    gate_stride = 0 if gate is None else _gate_stride(gate, M, H, dt)
    q, bs, y = out if out is not None else alloc_outputs(M, H, m, write_y, x)
    dev = x.get_device()
    n, w = 2 * M * H, 2 * H
    try:
        ok = (dev >= 0 and dev == _current_device() and x.is_contiguous()
              and residual.dtype is dt and residual.is_contiguous() and residual.nbytes >= n
              and residual.get_device() == dev
              and weight.dtype is dt and weight.is_contiguous() and weight.nbytes >= w and weight.get_device() == dev
              and (post_weight is None or (post_weight.dtype is dt and post_weight.is_contiguous()
                                           and post_weight.nbytes >= w and post_weight.get_device() == dev))
              and (residual_out is None or (residual_out.dtype is dt and residual_out.is_contiguous()
                                            and residual_out.nbytes >= n and residual_out.get_device() == dev))
              and (gate is None or gate.get_device() == dev)
              and _scale_ok(dev, m, scale) and _outputs_ok(dev, M, H, m, dt, write_y, q, bs, y))
    except AttributeError:
        ok = False
    if not ok:
        _need(x, "x", 0, (dt,))
        _need(residual, "residual", n, (dt,))
        if residual_out is not None:
            _need(residual_out, "residual_out", n, (dt,))
        if post_weight is not None:
            _need(post_weight, "post_weight", w, (dt,))
        _need(weight, "weight", w, (dt,))
        _need_scale(scale, "scale", m in (0, 1))
        _need_outputs(M, H, m, dt, write_y, (q, bs, y))
        dev = _place((x, residual, residual_out, post_weight, weight, gate, scale, q if m >= 0 else None,
                      bs if m > 0 else None, y if write_y else None))
    st = (_lib or load()).gemma_sandwich_norm_quant(
        x.data_ptr(), residual.data_ptr(), None if residual_out is None else residual_out.data_ptr(),
        None if post_weight is None else post_weight.data_ptr(), weight.data_ptr(),
        None if gate is None else gate.data_ptr(), gate_stride, float(residual_scale), float(eps),
        None if scale is None else scale.data_ptr(), m, 1 if write_y else 0, None if q is None else q.data_ptr(),
        None if bs is None else bs.data_ptr(), None if y is None else y.data_ptr(), M, H, _DTYPE[dt],
        _current_stream(dev) if stream is None else _stream(stream))
    if st:
        _check(st, "gemma_sandwich_norm_quant")
    return q, (scale if m == 0 else bs), (y if write_y else None)


def quantize(x, scale=None, mode="nvfp4", out=None, stream=None):
    """Codes and scales of a 16-bit matrix (dense rows, any row stride that is
    a multiple of 8): ``mode`` "fp8", "nvfp4" or "mxfp8".  ``out`` may supply
    (q, block_scale).  Returns (q, block_scale); for FP8 block_scale is
    ``scale`` itself."""
    m = _MODES[mode] if type(mode) is str else _mode(mode)
    if m < 0:
        raise ValueError("quantize needs a quantization mode")
    M, H, stride = _rows(x, "x")
    q, bs = out if out is not None else alloc_outputs(M, H, m, False, x)[:2]
    dev = x.get_device()
    try:
        ok = (dev >= 0 and dev == _current_device() and _scale_ok(dev, m, scale)
              and _outputs_ok(dev, M, H, m, None, False, q, bs, None))
    except AttributeError:
        ok = False
    if not ok:
        _need_scale(scale, "scale", m in (0, 1))
        _need_outputs(M, H, m, x.dtype, False, (q, bs, None))
        dev = _place((x, scale, q, bs if m > 0 else None))
    st = (_lib or load()).gnq_quantize(
        x.data_ptr(), stride, None if scale is None else scale.data_ptr(), m, q.data_ptr(),
        bs.data_ptr() if m > 0 else None, M, H, _DTYPE[x.dtype],
        _current_stream(dev) if stream is None else _stream(stream))
    if st:
        _check(st, "quantize")
    return q, (scale if m == 0 else bs)


def gated_act_quant(x, scale=None, mode="nvfp4", act="gelu_tanh", write_y=False, out=None, stream=None):
    """y = act(gate) * up for x = [gate | up] (M, 2H), quantized: the step
    between the two products of a gated MLP.  ``act`` is "silu" or
    "gelu_tanh"; ``mode`` "none" (y only), "fp8", "nvfp4" or "mxfp8"; ``out``
    may supply (q, block_scale, y).  Returns (q, block_scale, y)."""
    m = _MODES[mode] if type(mode) is str else _mode(mode)
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    M, W, stride = _rows(x, "x")
    if W % 2:
        raise ValueError("x must hold gate and up side by side: an even number of columns")
    H = W // 2
    write_y = bool(write_y) or m == -1
    q, bs, y = out if out is not None else alloc_outputs(M, H, m, write_y, x)
    dev = x.get_device()
    try:
        ok = (dev >= 0 and dev == _current_device() and _scale_ok(dev, m, scale)
              and _outputs_ok(dev, M, H, m, x.dtype, write_y, q, bs, y))
    except AttributeError:
        ok = False
    if not ok:
        _need_scale(scale, "scale", m in (0, 1))
        _need_outputs(M, H, m, x.dtype, write_y, (q, bs, y))
        dev = _place((x, scale, q if m >= 0 else None, bs if m > 0 else None, y if write_y else None))
    st = (_lib or load()).gated_act_quant(
        x.data_ptr(), stride, _ACTS[act], None if scale is None else scale.data_ptr(), m, 1 if write_y else 0,
        None if q is None else q.data_ptr(), None if bs is None else bs.data_ptr(),
        None if y is None else y.data_ptr(), M, H, _DTYPE[x.dtype],
        _current_stream(dev) if stream is None else _stream(stream))
    if st:
        _check(st, "gated_act_quant")
    return q, (scale if m == 0 else bs), (y if write_y else None)


def _packed(q, block_scale, name: str):
    """(rows, K) of packed NVFP4 codes with their swizzled block scales."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor of packed codes")
    M, half = q.shape
    _need(q, name, 0, (_U8,))
    _need(block_scale, name + "'s block scales", round_up(M, 128) * (half // 8), (_E4M3, _U8))
    return M, 2 * half


def _packed_ok(dev: int, q, sf) -> bool:
    M, half = q.shape
    return (q.dtype is _U8 and q.is_contiguous() and q.get_device() == dev and sf.dtype in (_E4M3, _U8)
            and sf.is_contiguous() and sf.nbytes >= (M + 127) // 128 * 16 * half and sf.get_device() == dev)


def nvfp4_dequantize(q, block_scale, scale=None, dtype=None, out=None, stream=None):
    """NVFP4 codes (M, K/2) and swizzled block scales back to values,
    code * (block scale / scale), as bf16 (default), fp16, fp32 or E4M3."""
    try:
        dev = q.get_device()
        M, half = q.shape
        K = 2 * half
        if out is None and dev >= 0:
            out = torch.empty((M, K), dtype=dtype or torch.bfloat16, device=q.device)
        ok = (dev >= 0 and dev == _current_device() and _packed_ok(dev, q, block_scale)
              and (scale is None or (scale.dtype is _F32 and scale.numel() == 1 and scale.get_device() == dev))
              and out.dtype in _OUT_TYPE and (dtype is None or out.dtype is dtype) and out.is_contiguous()
              and out.numel() >= M * K and out.get_device() == dev)
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        M, K = _packed(q, block_scale, "q")
        _need_scale(scale, "scale", False)
        if out is None:
            out = torch.empty((M, K), dtype=dtype or torch.bfloat16, pin_memory=True)
        if (not isinstance(out, torch.Tensor) or out.dtype not in _OUT_TYPE
                or (dtype is not None and out.dtype != dtype)):
            raise ValueError("the output must be bf16, fp16, fp32 or float8_e4m3fn (and of the given dtype)")
        _need(out, "out", M * K * out.element_size(), (out.dtype,))
        dev = _place((q, block_scale, scale, out))
    st = (_lib or load()).gnq_nvfp4_dequantize(
        q.data_ptr(), block_scale.data_ptr(), None if scale is None else scale.data_ptr(), out.data_ptr(), M, K,
        _OUT_TYPE[out.dtype], _current_stream(dev) if stream is None else _stream(stream))
    if st:
        _check(st, "nvfp4_dequantize")
    return out


def nvfp4_linear(q, block_scale, weight_q, weight_block_scale, alpha, bias=None, dtype=None, out=None,
                 stream=None):
    """alpha * (activation @ weight^T) + bias of NVFP4 operands: packed codes
    (M, K/2) and (N, K/2) with their swizzled block scales, as ``quantize``
    and the norm entry points return them.  ``alpha`` is a 1-element fp32
    tensor, usually 1 / (scale of the activation * scale of the weight).
    The output (M, N) is bf16 (default), fp16 or fp32."""
    try:
        dev = q.get_device()
        M, half = q.shape
        N, wide = weight_q.shape
        K = 2 * half
        if out is None:
            out = torch.empty((M, N), dtype=dtype or torch.bfloat16, device=q.device)
        ot = _OUT_TYPE.get(out.dtype, 3)
        ok = (ot < 3 and wide == half and dev >= 0 and dev == _current_device()
              and (dtype is None or out.dtype is dtype)
              and _packed_ok(dev, q, block_scale) and _packed_ok(dev, weight_q, weight_block_scale)
              and alpha.dtype is _F32 and alpha.numel() == 1 and alpha.get_device() == dev
              and out.is_contiguous() and out.numel() >= M * N and out.get_device() == dev
              and (bias is None or (ot < 2 and bias.dtype is out.dtype and bias.is_contiguous() and bias.numel() >= N
                                    and bias.get_device() == dev)))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        M, K = _packed(q, block_scale, "q")
        N, Kw = _packed(weight_q, weight_block_scale, "weight_q")
        if K != Kw:
            raise ValueError(f"the activation has K = {K}, the weight {Kw}")
        _need_scale(alpha, "alpha", True)
        ot = _OUT_TYPE.get(out.dtype, 3) if isinstance(out, torch.Tensor) else 3
        if ot == 3 or (dtype is not None and out.dtype != dtype):
            raise ValueError("the output must be bf16, fp16 or fp32 (and of the given dtype)")
        _need(out, "out", M * N * out.element_size(), (out.dtype,))
        if bias is not None:
            _need(bias, "bias", N * 2, (out.dtype,) if ot < 2 else (torch.bfloat16, torch.float16))
        dev = _place((q, block_scale, weight_q, weight_block_scale, alpha, bias, out), pinned=False)
    st = (_lib or load()).nvfp4_linear(
        q.data_ptr(), block_scale.data_ptr(), weight_q.data_ptr(), weight_block_scale.data_ptr(), alpha.data_ptr(),
        None if bias is None else bias.data_ptr(), out.data_ptr(), M, N, K, ot,
        0 if bias is None else _DTYPE.get(bias.dtype, 2), _current_stream(dev) if stream is None else _stream(stream))
    if st:
        _check(st, "nvfp4_linear")
    return out


def set_launch_policy(kernel: int = 0, cluster: int = 0, vpt: int = 0, form: int = 0) -> None:
    """Force the launch shape (0 = automatic): kernel 1 = row kernel, 2 =
    streaming kernel; cluster = CTAs per row; vpt = units per thread; form
    1 = fp32 (fewest instructions), 2 = packed (fewest registers)."""
    _check(load().gnq_set_launch_policy(int(kernel), int(cluster), int(vpt), int(form)),
           "gnq_set_launch_policy")


def query_launch(M: int, H: int, mode, dtype: str = "bf16", k: int = 1, residual: bool = True,
                 write_y: bool = False, weight_bias: float = 1.0) -> tuple[int, int, int, int]:
    """The automatic launch shape of a call, as (kernel, cluster, vpt, form) in
    set_launch_policy's terms; forcing it reproduces the automatic launch."""
    out = [ctypes.c_int(0) for _ in range(4)]
    dt = {"bf16": 0, "fp16": 1}[dtype] if isinstance(dtype, str) else _DTYPE[dtype]
    _check(load().gnq_query_launch(int(M), int(H), int(k), int(bool(residual)), int(bool(write_y)),
                                   _mode(mode), dt, float(weight_bias),
                                   *[ctypes.byref(o) for o in out]), "gnq_query_launch")
    return tuple(o.value for o in out)


def set_linear_policy(kernel: int = 0) -> None:
    """Force the kernel of later nvfp4_linear calls (0 = automatic): 1 = tiles
    of one CTA with a split K, 2 = CTA pairs on 256 x 256 tiles."""
    _check(load().gnq_set_linear_policy(int(kernel)), "gnq_set_linear_policy")


def query_linear(M: int, N: int, K: int, dtype=torch.bfloat16) -> tuple[int, int, int]:
    """(kernel, tokens of a tile, CTAs that share a tile's K) that nvfp4_linear
    picks by itself, in set_linear_policy's terms."""
    out = [ctypes.c_int(0) for _ in range(3)]
    _check(load().gnq_query_linear(int(M), int(N), int(K), _OUT_TYPE[dtype], *[ctypes.byref(o) for o in out]),
           "gnq_query_linear")
    return tuple(o.value for o in out)


def set_pdl(enable: bool) -> None:
    """Programmatic dependent launch on (default) or off for later calls."""
    _check(load().gnq_set_pdl(1 if enable else 0), "gnq_set_pdl")


def pdl_consumer(q: torch.Tensor, wt: torch.Tensor, out: torch.Tensor, ctas: int,
                 stream=None) -> None:
    """Diagnostic stand-in for the next layer's first kernel: reads wt, waits
    on the preceding kernel, reads q, writes ctas * 256 checksum words."""
    for t, name in ((q, "q"), (wt, "wt")):
        if not (t.is_cuda and t.is_contiguous() and (t.numel() * t.element_size()) % 16 == 0):
            raise ValueError(f"{name} must be a contiguous CUDA tensor of whole 16-byte units")
    if not (out.is_cuda and out.dtype == torch.int32 and out.numel() >= ctas * 256):
        raise ValueError("out must be an int32 CUDA tensor of at least ctas * 256 words")
    _check(load().gnq_pdl_consumer(_ptr(q), q.numel() * q.element_size(), _ptr(wt),
                                   wt.numel() * wt.element_size(), _ptr(out), int(ctas),
                                   _stream(stream)), "gnq_pdl_consumer")


def set_constant_weights(enable: bool) -> None:
    """Read w and the scale before waiting on the preceding kernel (the caller
    guarantees no preceding kernel writes them); off by default."""
    _check(load().gnq_set_constant_weights(1 if enable else 0), "gnq_set_constant_weights")


def inject_wait_timeout(enable: bool) -> None:
    """Test hook: later streaming launches make their bounded waits give up
    (device error bit 1, no outputs written); off by default."""
    _check(load().gnq_inject_wait_timeout(1 if enable else 0), "gnq_inject_wait_timeout")


def inject_split_timeout(cta: int = -1) -> None:
    """Test hook: CTA ``cta`` (0..7) of each cluster of later split products
    gives up, alone (device error bit 1, no outputs written); -1 turns it off."""
    _check(load().gnq_inject_split_timeout(int(cta)), "gnq_inject_split_timeout")


def read_device_error(clear: bool = True) -> int:
    """The device error word (bit 1: a bounded wait in a kernel gave up)."""
    flags = ctypes.c_uint(0)
    _check(load().gnq_read_device_error(ctypes.byref(flags), 1 if clear else 0),
           "gnq_read_device_error")
    return int(flags.value)


def quantize_fp8_values(y: torch.Tensor, scale: torch.Tensor, stream=None) -> torch.Tensor:
    """The kernels' static-FP8 quantizer on raw fp32 values (diagnostic)."""
    if not (y.is_cuda and y.dtype == torch.float32 and y.is_contiguous()):
        raise ValueError("y must be a contiguous fp32 CUDA tensor")
    q = torch.empty(y.shape, dtype=torch.uint8, device=y.device)
    _check(load().gnq_quantize_fp8_values(_ptr(y), y.numel(), _scale_ptr(scale), _ptr(q),
                                          _stream(stream)), "gnq_quantize_fp8_values")
    return q


def encode_e4m3_e2m1(v: torch.Tensor, stream=None):
    """Hardware E4M3 and E2M1 codes of fp32 values (diagnostic)."""
    if not (v.is_cuda and v.dtype == torch.float32 and v.is_contiguous()):
        raise ValueError("v must be a contiguous fp32 CUDA tensor")
    e4 = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    e2 = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check(load().gnq_encode_e4m3_e2m1(_ptr(v), v.numel(), _ptr(e4), _ptr(e2), _stream(stream)),
           "gnq_encode_e4m3_e2m1")
    return e4, e2
