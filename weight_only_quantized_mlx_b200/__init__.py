"""Python binding of libmlxq.so, the B200 (sm_100a) library for the 8-bit
group-affine quantized linear layer of the "MlxInt8Weight" API page.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  The functions carry the C names of ``include/mlxq.h``; buffers may be
given as torch tensors (their ``data_ptr()`` is passed) or as raw integer
device addresses, streams as ``torch.cuda.Stream`` objects, raw integers or
``None`` (torch's current stream).  A nonzero status raises :class:`MlxqError`.

There is no CPU fallback: importing the binding without the built library
raises ``ImportError`` (build it with ``python -m
weight_only_quantized_mlx_b200.build``).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmlxq.so")

MLXQ_OK = 0
MLXQ_ERR_INVALID_ARG = 1
MLXQ_ERR_PARSE = 2
MLXQ_ERR_MISSING_TENSOR = 3
MLXQ_ERR_DTYPE = 4
MLXQ_ERR_SHAPE = 5
MLXQ_ERR_GROUP_SIZE = 6
MLXQ_ERR_UNSUPPORTED = 7
MLXQ_ERR_CUDA = 8
MLXQ_ERR_DEVICE_TIMEOUT = 9

MLXQ_GEMM_AUTO = 0
MLXQ_GEMM_ROWS = 1
MLXQ_GEMM_SMALLM = 2
MLXQ_GEMM_TCGEN05 = 3
MLXQ_GEMM_SMALLM_FFMA = 4
MLXQ_GEMM_SMALLM_GROUPS = 5
MLXQ_GEMM_SMALLM_TC = 6

MLXQ_WEIGHT_STATIC = 1

MLXQ_MOE_SOFTMAX_ALL = 1

MLXQ_DTYPE_BF16 = 0
MLXQ_DTYPE_F16 = 1
MLXQ_DTYPE_F32 = 2

EXPORTS = ("mlxq_load", "mlxq_dequant", "mlxq_gemv", "mlxq_gemv_silu_gate",
           "mlxq_gemv_silu_gate_resid", "mlxq_gemm", "mlxq_gemm_with", "mlxq_gemm_noalloc", "mlxq_release",
           "mlxq_last_error", "mlxq_device_status", "mlxq_dequant_as", "mlxq_quantize", "mlxq_selftest_wait_timeout",
           "mlxq_selftest_fail_alloc", "mlxq_mx4_quantize", "mlxq_mx4_dequant", "mlxq_mx4_gemm", "mlxq_mx4_matmul",
           "mlxq_moe_workspace_bytes", "mlxq_moe", "mlxq_mx4_moe")


class mlxq_weight(ctypes.Structure):
    """C ``mlxq_weight``: three device pointers and the dimensions.  A handle made by
    :func:`weight_view` keeps its tensors alive (``tensors``); ``problem`` says why
    they are not a whole weight, where they are not."""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("out_features", ctypes.c_uint32),
                ("in_features", ctypes.c_uint32), ("group_size", ctypes.c_uint32),
                ("flags", ctypes.c_uint32)]
    tensors = None
    problem = None


class mlxq_mx4(ctypes.Structure):
    """C ``mlxq_mx4``: codes and scales of an MX4 matrix.  A handle made by
    :func:`mx4_view` or :func:`mx4_empty` keeps its tensors alive (``tensors``)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_uint32), ("cols", ctypes.c_uint32)]
    tensors = None


class MlxqError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"mlxq error {code}: {message}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run python -m weight_only_quantized_mlx_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        W = ctypes.POINTER(mlxq_weight)
        Q = ctypes.POINTER(mlxq_mx4)
        vp, u64, u32, i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int
        sigs = {
            "mlxq_load": [ctypes.c_char_p, ctypes.c_size_t, ctypes.c_char_p, u32, W],
            "mlxq_dequant": [W, vp, u64],
            "mlxq_gemv": [W, vp, vp, u64],
            "mlxq_gemv_silu_gate": [W, vp, vp, vp, u64],
            "mlxq_gemv_silu_gate_resid": [W, vp, vp, vp, vp, u64],
            "mlxq_gemm": [W, vp, vp, u32, u64],
            "mlxq_gemm_with": [W, vp, vp, u32, i32, u64],
            "mlxq_gemm_noalloc": [W, vp, vp, u32, u64],
            "mlxq_release": [W],
            "mlxq_last_error": [],
            "mlxq_device_status": [],
            "mlxq_quantize": [vp, W, u64],
            "mlxq_dequant_as": [W, vp, i32, u64],
            "mlxq_selftest_wait_timeout": [u32, u64],
            "mlxq_selftest_fail_alloc": [u32],
            "mlxq_mx4_quantize": [vp, Q, u64],
            "mlxq_mx4_dequant": [Q, vp, u64],
            "mlxq_mx4_gemm": [Q, vp, vp, u32, u64],
            "mlxq_mx4_matmul": [Q, Q, vp, u64],
            "mlxq_moe_workspace_bytes": [u32, u32, u32, u32],
            "mlxq_moe": [vp, W, W, W, u32, u32, u32, vp, vp, u32, vp, ctypes.c_size_t, u64],
            "mlxq_mx4_moe": [vp, Q, Q, Q, u32, u32, u32, vp, vp, u32, vp, ctypes.c_size_t, u64],
        }
        returns = {"mlxq_last_error": ctypes.c_char_p, "mlxq_moe_workspace_bytes": ctypes.c_size_t}
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = returns.get(name, ctypes.c_int)
        _lib = L
    return _lib


def _ptr(b):
    if b is None:
        return None
    if isinstance(b, int):
        return b
    return b.data_ptr()


_raw_stream = None


def _find_raw_stream():
    """A function from a device to torch's current stream there, as an integer.
    Without building a Stream object where torch has the shortcut: 0.5 against
    4.4 us a call, of the 10 us that a small call took."""
    global _raw_stream
    import torch
    if not torch.cuda.is_available():
        return lambda device: 0
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is None:
        _raw_stream = lambda device: torch.cuda.current_stream(device).cuda_stream
    return _raw_stream


def _stream(s, device=None) -> int:
    if s is None:
        return (_raw_stream or _find_raw_stream())(_device() if device is None else device)
    if isinstance(s, int):
        return s
    return s.cuda_stream


_current_device = None


def _device() -> int:
    """torch's current device, -1 where there is none."""
    global _current_device
    if _current_device is None:
        import torch
        if not torch.cuda.is_available():
            return -1
        torch.cuda.init()
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _current_device()


def _local(b, name: str, device: int) -> None:
    """Refuse a tensor that is not on the current device: a kernel must not get its address."""
    if b.get_device() != device:
        raise MlxqError(MLXQ_ERR_INVALID_ARG, f"{name} is on {b.device}, the current device is cuda:{device}")


_bf16 = None  # torch.bfloat16, once it has been seen


def _dense(b, name: str, elems: int, device: int):
    """The address of a buffer that holds `elems` contiguous BF16 elements on the
    current device; raw addresses are taken as they are."""
    global _bf16
    if b is None or isinstance(b, int):
        return b
    if _bf16 is None and str(b.dtype) == "torch.bfloat16":
        _bf16 = b.dtype
    if b.dtype is not _bf16 or not b.is_contiguous() or b.numel() < elems:
        raise MlxqError(MLXQ_ERR_INVALID_ARG, f"{name} must be a contiguous bfloat16 tensor of at least {elems} elements, "
                                              f"got {b.dtype} {tuple(b.shape)} with strides {tuple(b.stride())}")
    if b.get_device() != device:
        _local(b, name, device)
    return b.data_ptr()


def _fits(**numbers) -> None:
    """Refuse numbers that 32 bits do not hold: ctypes would cut them to others."""
    for name, v in numbers.items():
        if not 0 <= v <= 0xFFFFFFFF:
            raise MlxqError(MLXQ_ERR_INVALID_ARG, f"{name} is out of range: {v}")


def _mx4(h: mlxq_mx4, name: str, device: int):
    """A handle as an argument of a call; its tensors, where it has any, are on the current device."""
    if h.tensors is not None and h.tensors[0].get_device() != device:
        _local(h.tensors[0], name, device)
    return ctypes.byref(h)


def _q8(h: mlxq_weight, name: str, device: int):
    """The same for an 8-bit handle."""
    if h.tensors is not None:
        if h.problem is not None:
            raise MlxqError(MLXQ_ERR_INVALID_ARG, f"{name}: {h.problem}")
        if h.tensors[0].get_device() != device:
            _local(h.tensors[0], name, device)
    return ctypes.byref(h)


def _check(rc: int) -> None:
    if rc != MLXQ_OK:
        raise MlxqError(rc, mlxq_last_error())


def mlxq_last_error() -> str:
    return lib().mlxq_last_error().decode(errors="replace")


def mlxq_load(blob: bytes, base: str, group_size: int) -> mlxq_weight:
    w = mlxq_weight()
    _check(lib().mlxq_load(blob, len(blob), base.encode(), group_size, ctypes.byref(w)))
    return w


def mlxq_release(w: mlxq_weight) -> None:
    _check(lib().mlxq_release(ctypes.byref(w)))


def mlxq_dequant(w: mlxq_weight, out, stream=None) -> None:
    _check(lib().mlxq_dequant(ctypes.byref(w), _ptr(out), _stream(stream)))


def mlxq_gemv(w: mlxq_weight, x, y, stream=None) -> None:
    _check(lib().mlxq_gemv(ctypes.byref(w), _ptr(x), _ptr(y), _stream(stream)))


def mlxq_gemv_silu_gate(w: mlxq_weight, gate, up, y, stream=None) -> None:
    _check(lib().mlxq_gemv_silu_gate(ctypes.byref(w), _ptr(gate), _ptr(up), _ptr(y), _stream(stream)))


def mlxq_gemv_silu_gate_resid(w: mlxq_weight, gate, up, x_resid, y, stream=None) -> None:
    _check(lib().mlxq_gemv_silu_gate_resid(ctypes.byref(w), _ptr(gate), _ptr(up), _ptr(x_resid),
                                           _ptr(y), _stream(stream)))


def mlxq_gemm(w: mlxq_weight, x, y, m: int, stream=None) -> None:
    _check(lib().mlxq_gemm(ctypes.byref(w), _ptr(x), _ptr(y), m, _stream(stream)))


def mlxq_gemm_with(w: mlxq_weight, x, y, m: int, kernel: int, stream=None) -> None:
    _check(lib().mlxq_gemm_with(ctypes.byref(w), _ptr(x), _ptr(y), m, kernel, _stream(stream)))


def mlxq_gemm_noalloc(w: mlxq_weight, x, y, m: int, stream=None) -> None:
    _check(lib().mlxq_gemm_noalloc(ctypes.byref(w), _ptr(x), _ptr(y), m, _stream(stream)))


MLXQ_STATIC_SCRATCH_BYTES = 40 << 20


def mlxq_device_status() -> None:
    _check(lib().mlxq_device_status())


def mlxq_dequant_as(w: mlxq_weight, out, dtype: int, stream=None) -> None:
    _check(lib().mlxq_dequant_as(ctypes.byref(w), _ptr(out), dtype, _stream(stream)))


def mlxq_quantize(w_bf16, dst: mlxq_weight, stream=None) -> None:
    _check(lib().mlxq_quantize(_ptr(w_bf16), ctypes.byref(dst), _stream(stream)))


def mlxq_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _check(lib().mlxq_selftest_wait_timeout(limit_us, _stream(stream)))


def mlxq_selftest_fail_alloc(nth: int) -> None:
    _check(lib().mlxq_selftest_fail_alloc(nth))


def weight_view(packed, scales, biases, group_size: int, flags: int = 0) -> mlxq_weight:
    """A non-owning handle over caller-owned device tensors (packed uint32/int32
    [N, K/4], scales/biases bf16 [N, K/gs]).  Never pass it to mlxq_release."""
    N = packed.shape[0]
    K = packed.shape[1] * 4
    h = mlxq_weight(_ptr(packed), _ptr(scales), _ptr(biases), N, K, group_size, flags)
    tensors = (packed, scales, biases)
    if all(hasattr(t, "get_device") for t in tensors):
        h.tensors = tensors
        h.problem = _weight_problem(packed, scales, biases, group_size)
    return h


def _weight_problem(packed, scales, biases, group_size: int):
    """Why tensors are not a contiguous weight in one place (None: they are)."""
    if not all(t.is_contiguous() for t in (packed, scales, biases)):
        return "packed, scales and biases must be contiguous"
    if packed.dim() != 2 or packed.element_size() != 4:
        return f"packed must be 32-bit [N, K/4], got {packed.dtype} {tuple(packed.shape)}"
    if max(packed.shape[0], packed.shape[1] * 4) > 0xFFFFFFFF:
        return f"dimensions must fit 32 bits, got {packed.shape[0]} x {packed.shape[1] * 4}"
    for t in (scales, biases):
        if str(t.dtype) != "torch.bfloat16" or t.numel() * group_size != packed.numel() * 4:
            return f"scales and biases must be bfloat16 [N, K/{group_size}], got {t.dtype} {tuple(t.shape)}"
        if t.device != packed.device:
            return f"packed is on {packed.device} and its tables on {t.device}"
    return None


def mx4_view(codes, scales) -> mlxq_mx4:
    """A handle over device tensors: codes (u)int32 [rows, cols/8], scales uint8
    [rows, cols/32], both contiguous."""
    if codes.dim() != 2 or scales.dim() != 2 or codes.element_size() != 4 or scales.element_size() != 1 \
            or tuple(scales.shape) != (codes.shape[0], codes.shape[1] // 4) or codes.shape[1] % 4:
        raise MlxqError(MLXQ_ERR_SHAPE, f"MX4 codes must be 32-bit [rows, cols/8] and scales 8-bit [rows, cols/32], got "
                                        f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise MlxqError(MLXQ_ERR_INVALID_ARG, "MX4 codes and scales must be contiguous")
    if max(codes.shape[0], codes.shape[1] * 8) > 0xFFFFFFFF:
        raise MlxqError(MLXQ_ERR_SHAPE, f"MX4 dimensions must fit 32 bits, got {codes.shape[0]} x {codes.shape[1] * 8}")
    if codes.device != scales.device:
        raise MlxqError(MLXQ_ERR_INVALID_ARG, f"MX4 codes are on {codes.device} and scales on {scales.device}")
    h = mlxq_mx4(_ptr(codes), _ptr(scales), codes.shape[0], codes.shape[1] * 8)
    h.tensors = (codes, scales)
    return h


def mx4_empty(rows: int, cols: int, device="cuda") -> mlxq_mx4:
    """A handle over new, unfilled tensors, as a destination of mlxq_mx4_quantize."""
    import torch
    if cols % 32:
        raise MlxqError(MLXQ_ERR_SHAPE, f"cols {cols} is not a multiple of 32")
    return mx4_view(torch.empty(rows, cols // 8, dtype=torch.int32, device=device),
                    torch.empty(rows, cols // 32, dtype=torch.uint8, device=device))


def mlxq_mx4_quantize(x_bf16, dst: mlxq_mx4, stream=None) -> None:
    d = _device()
    x = _dense(x_bf16, "x", dst.rows * dst.cols, d)
    _check(lib().mlxq_mx4_quantize(x, _mx4(dst, "dst", d), _stream(stream, d)))


def mlxq_mx4_dequant(w: mlxq_mx4, out, stream=None) -> None:
    d = _device()
    out = _dense(out, "out", w.rows * w.cols, d)
    _check(lib().mlxq_mx4_dequant(_mx4(w, "w", d), out, _stream(stream, d)))


def mlxq_mx4_gemm(w: mlxq_mx4, x, y, m: int, stream=None) -> None:
    d = _device()
    _fits(m=m)
    x, y = _dense(x, "X", m * w.cols, d), _dense(y, "Y", m * w.rows, d)
    _check(lib().mlxq_mx4_gemm(_mx4(w, "w", d), x, y, m, _stream(stream, d)))


def mlxq_mx4_matmul(w: mlxq_mx4, a: mlxq_mx4, y, stream=None) -> None:
    d = _device()
    y = _dense(y, "Y", a.rows * w.rows, d)
    _check(lib().mlxq_mx4_matmul(_mx4(w, "w", d), _mx4(a, "a", d), y, _stream(stream, d)))


def mlxq_moe_workspace_bytes(hidden: int, inter: int, top_k: int, m: int) -> int:
    if not all(0 <= v <= 0xFFFFFFFF for v in (hidden, inter, top_k, m)):
        return 0
    return lib().mlxq_moe_workspace_bytes(hidden, inter, top_k, m)


def _moe(fn, hidden, router, weights, experts, top_k, x, y, m, workspace, stream, flags, d):
    _fits(experts=experts, top_k=top_k, m=m, flags=flags)
    router = _dense(router, "router", experts * hidden, d)
    x, y = _dense(x, "x", m * hidden, d), _dense(y, "y", m * hidden, d)
    if not hasattr(workspace, "data_ptr") or not workspace.is_contiguous():
        raise MlxqError(MLXQ_ERR_INVALID_ARG, "workspace must be a contiguous tensor")
    if hasattr(workspace, "get_device"):
        _local(workspace, "workspace", d)
    _check(fn(router, *weights, experts, top_k, flags, x, y, m, workspace.data_ptr(),
              workspace.numel() * workspace.element_size(), _stream(stream, d)))


def mlxq_moe(router, gate: mlxq_weight, up: mlxq_weight, down: mlxq_weight, experts: int, top_k: int, x, y, m: int,
             workspace, stream=None, flags: int = 0) -> None:
    """workspace: a device tensor of at least mlxq_moe_workspace_bytes(...) bytes, for one call at a time."""
    d = _device()
    weights = [_q8(gate, "gate", d), _q8(up, "up", d), _q8(down, "down", d)]
    _moe(lib().mlxq_moe, gate.in_features, router, weights, experts, top_k, x, y, m, workspace, stream, flags, d)


def mlxq_mx4_moe(router, gate: mlxq_mx4, up: mlxq_mx4, down: mlxq_mx4, experts: int, top_k: int, x, y, m: int,
                 workspace, stream=None, flags: int = 0) -> None:
    """workspace: a device tensor of at least mlxq_moe_workspace_bytes(...) bytes, for one call at a time."""
    d = _device()
    weights = [_mx4(gate, "gate", d), _mx4(up, "up", d), _mx4(down, "down", d)]
    _moe(lib().mlxq_mx4_moe, gate.cols, router, weights, experts, top_k, x, y, m, workspace, stream, flags, d)


class MlxInt8Weight:
    """The page's struct as a Python object: ``load`` / ``dequantize_to`` /
    ``gemv`` / ``gemv_silu_gate`` / ``gemv_silu_gate_resid`` / ``gemm`` /
    ``release``, each one call into the C ABI."""

    def __init__(self, handle: mlxq_weight, owned: bool):
        self.handle = handle
        self.owned = owned

    @classmethod
    def load(cls, blob: bytes, base: str, group_size: int, static: bool = False) -> "MlxInt8Weight":
        """static=True sets MLXQ_WEIGHT_STATIC (see include/mlxq.h): the caller
        promises that no kernel writes the weight while calls read it."""
        w = cls(mlxq_load(blob, base, group_size), True)
        if static:
            w.handle.flags |= MLXQ_WEIGHT_STATIC
        return w

    @property
    def out_features(self) -> int:
        return self.handle.out_features

    @property
    def in_features(self) -> int:
        return self.handle.in_features

    @property
    def group_size(self) -> int:
        return self.handle.group_size

    def dequantize_to(self, out, stream=None):
        mlxq_dequant(self.handle, out, stream)

    def gemv(self, x, y, stream=None):
        mlxq_gemv(self.handle, x, y, stream)

    def gemv_silu_gate(self, gate, up, y, stream=None):
        mlxq_gemv_silu_gate(self.handle, gate, up, y, stream)

    def gemv_silu_gate_resid(self, gate, up, x_resid, y, stream=None):
        mlxq_gemv_silu_gate_resid(self.handle, gate, up, x_resid, y, stream)

    def gemm(self, x, y, m: int, stream=None):
        mlxq_gemm(self.handle, x, y, m, stream)

    def release(self):
        if not self.owned:
            raise MlxqError(MLXQ_ERR_INVALID_ARG, "this handle does not own its buffers")
        mlxq_release(self.handle)
