"""Python binding of libqz.so, the B200 weight-only quantization library.

Argument marshalling only: every function below validates Python-side types,
allocates outputs with PyTorch when the caller did not pass them, and calls
the C entry point of the same name (declared in ``include/qz.h``) on the
``stream`` argument, else the current CUDA stream; outputs and temporary
workspaces are allocated on that same stream.  All arithmetic runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback.  If ``libqz.so``
is missing the import fails.
"""
import contextlib
import ctypes
import os

import torch

__all__ = [
    "QzError", "lib", "qz_version", "qz_status_string", "qz_packed_bytes",
    "qz_workspace_bytes", "qz_workspace_bytes_for_sms", "qz_quantize_pack", "qz_dequantize",
    "qz_w4a16_gemv",
    "qz_w4a16_gemm", "qz_w8a16_gemv", "qz_w8a16_gemm", "qz_set_device_wait_limit",
    "qz_set_launch_overlap", "qz_device_status", "qz_gptq_quantize", "QZ_OP_GPTQ",
    "qz_fp4_packed_bytes", "qz_fp4_quantize", "qz_fp4_dequantize", "qz_fp4a16_gemv",
    "QZ_OP_FP4A16_GEMV", "QZ_FP4_MX", "QZ_FP4_NV", "qz_fp4_mma_scale_bytes",
    "qz_fp4_scales_to_mma", "qz_fp4a4_gemm", "QZ_OP_FP4A4_GEMM",
    "qz_kv4_cache_bytes", "qz_kv4_append", "qz_kv4_read", "qz_kv4_attention",
    "QZ_OP_KV4_ATTENTION", "qz_w4a16_lora_gemv", "qz_w8a16_lora_gemv", "QZ_OP_W4A16_LORA_GEMV",
    "QZ_OP_W8A16_LORA_GEMV",
    "Workspace", "QZ_WORKSPACE_COUNTERS", "QZ_OP_QUANTIZE_PACK", "QZ_OP_DEQUANTIZE", "QZ_OP_W4A16_GEMV",
    "QZ_OP_W4A16_GEMM", "QZ_OP_W8A16_GEMV", "QZ_OP_W8A16_GEMM", "EXPORTED_SYMBOLS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqz.so")

QZ_OK = 0
QZ_ERR_DEVICE_TIMEOUT = 6
QZ_ERR_DEVICE_INDEX = 7
(QZ_OP_QUANTIZE_PACK, QZ_OP_DEQUANTIZE, QZ_OP_W4A16_GEMV, QZ_OP_W4A16_GEMM, QZ_OP_W8A16_GEMV,
 QZ_OP_W8A16_GEMM, QZ_OP_GPTQ, QZ_OP_FP4A16_GEMV, QZ_OP_FP4A4_GEMM,
 QZ_OP_KV4_ATTENTION, QZ_OP_W4A16_LORA_GEMV, QZ_OP_W8A16_LORA_GEMV) = range(12)
QZ_FP4_MX, QZ_FP4_NV = 0, 1
QZ_WORKSPACE_COUNTERS = 8192
FP4_BLOCK = {QZ_FP4_MX: 32, QZ_FP4_NV: 16}

_i32, _i64, _sz, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
_f32 = ctypes.c_float
_SIGS = {
    "qz_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "qz_version": ([], ctypes.c_int),
    "qz_packed_bytes": ([_i64, _i64, _i32, _i32, _i64, ctypes.POINTER(_sz),
                         ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "qz_workspace_bytes": ([_i32, _i64, _i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "qz_workspace_bytes_for_sms": ([_i32, _i64, _i64, _i64, _i64, _i32, ctypes.POINTER(_sz)],
                                   ctypes.c_int),
    "qz_quantize_pack": ([_p, _i64, _i64, _i32, _i32, _i64, _p, _p, _p, _p, _sz, _p], ctypes.c_int),
    "qz_dequantize": ([_p, _p, _p, _i64, _i64, _i32, _i32, _i64, _p, _p], ctypes.c_int),
    "qz_w4a16_gemv": ([_p, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _p, _sz, _p], ctypes.c_int),
    "qz_w4a16_gemm": ([_p, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _p, _sz, _p], ctypes.c_int),
    "qz_w8a16_gemv": ([_p, _p, _p, _i64, _i64, _i64, _p, _p, _sz, _p], ctypes.c_int),
    "qz_w8a16_gemm": ([_p, _p, _p, _i64, _i64, _i64, _p, _p, _sz, _p], ctypes.c_int),
    "qz_w4a16_gemv_noalloc": ([_p, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _p], ctypes.c_int),
    "qz_gptq_quantize": ([_p, _p, _i64, _i64, _i64, _i32, _i32, _i64, ctypes.c_double, _p, _p, _p,
                          _p, _sz, _p], ctypes.c_int),
    "qz_fp4_packed_bytes": ([_i64, _i64, _i32, ctypes.POINTER(_sz), ctypes.POINTER(_sz)],
                            ctypes.c_int),
    "qz_fp4_quantize": ([_p, _i64, _i64, _i32, _p, _p, _p, _p], ctypes.c_int),
    "qz_fp4_dequantize": ([_p, _p, _p, _i64, _i64, _i32, _p, _p], ctypes.c_int),
    "qz_fp4a16_gemv": ([_p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _p, _sz, _p], ctypes.c_int),
    "qz_fp4_mma_scale_bytes": ([_i64, _i64, _i32, ctypes.POINTER(_sz)], ctypes.c_int),
    "qz_fp4_scales_to_mma": ([_p, _i64, _i64, _i32, _p, _p], ctypes.c_int),
    "qz_fp4a4_gemm": ([_p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _p, _sz, _p], ctypes.c_int),
    "qz_w4a16_lora_gemv": ([_p] * 4 + [_i64] * 4 + [_p] * 4 + [_i64] * 2 + [_p, _p, _sz, _p],
                           ctypes.c_int),
    "qz_w8a16_lora_gemv": ([_p] * 3 + [_i64] * 3 + [_p] * 4 + [_i64] * 2 + [_p, _p, _sz, _p],
                           ctypes.c_int),
    "qz_kv4_cache_bytes": ([_i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "qz_kv4_append": ([_p, _p, _p, _i64, _i64, _p, _p, _p] + [_i64] * 8 + [_p], ctypes.c_int),
    "qz_kv4_read": ([_p, _p, _p, _p] + [_i64] * 8 + [_p, _p, _p], ctypes.c_int),
    "qz_kv4_attention": ([_p, _i64, _p, _p, _p, _p] + [_i64] * 9 + [_f32, _i64, _p, _i64, _p, _sz,
                                                                    _p], ctypes.c_int),
    "qz_set_device_wait_limit": ([ctypes.c_uint64], None),
    "qz_set_launch_overlap": ([ctypes.c_int32], ctypes.c_int),
    "qz_device_status": ([], ctypes.c_int),
}
EXPORTED_SYMBOLS = tuple(_SIGS)

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python weight_only_quantization_wise_b200/build.py` "
        "(there is no fallback implementation)")

lib = ctypes.CDLL(LIB_PATH)
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class QzError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {qz_status_string(status)} (status {status})")


def _check(status: int, where: str) -> None:
    if status != QZ_OK:
        raise QzError(status, where)


def qz_status_string(status: int) -> str:
    return lib.qz_status_string(int(status)).decode()


def qz_version() -> int:
    return int(lib.qz_version())


def qz_packed_bytes(N, K, bits=4, symmetric=False, group_size=128):
    c, s, z = _sz(), _sz(), _sz()
    _check(lib.qz_packed_bytes(N, K, bits, int(symmetric), group_size, ctypes.byref(c),
                               ctypes.byref(s), ctypes.byref(z)), "qz_packed_bytes")
    return c.value, s.value, z.value


_WS_SIZES = {}


def qz_workspace_bytes(op, M, N, K, group_size=128) -> int:
    """Workspace bytes of a call (a pure function of the arguments; cached)."""
    key = (int(op), int(M), int(N), int(K), int(group_size))
    v = _WS_SIZES.get(key)
    if v is None:
        b = _sz()
        _check(lib.qz_workspace_bytes(*key, ctypes.byref(b)), "qz_workspace_bytes")
        v = _WS_SIZES[key] = b.value
    return v


def qz_workspace_bytes_for_sms(op, M, N, K, group_size, sms) -> int:
    """Workspace bytes of a call whose grid is sized for `sms` SMs."""
    b = _sz()
    _check(lib.qz_workspace_bytes_for_sms(int(op), int(M), int(N), int(K), int(group_size),
                                          int(sms), ctypes.byref(b)), "qz_workspace_bytes_for_sms")
    return b.value


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _launch_stream(stream, device):
    """The torch stream a call runs on: `stream`, else the current stream."""
    return torch.cuda.current_stream(device) if stream is None else stream


def _on(stream):
    """Context that makes an explicitly passed stream current for the call's
    allocations (nothing to do when the call runs on the current stream)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _handle(stream):
    return ctypes.c_void_p(stream.cuda_stream)


class Workspace:
    """Device workspaces that grow on demand; one serves every call issued on
    one stream.

    Each call leaves the counters in its workspace at zero again; the rest is
    scratch that every call writes before it reads.  The split-K calls of every
    size share one buffer, which is QZ_WORKSPACE_COUNTERS bytes larger than any
    of them needs (their counters lie in its last bytes); `key` names the
    zero-filled buffers of calls that keep their counters elsewhere.  A buffer
    that a captured graph uses is kept when a larger one takes its place.
    Calls that may run concurrently need separate Workspace objects.
    """

    def __init__(self, device=None):
        self.device = torch.device(device if device is not None else "cuda")
        self.bufs = {}
        self.captured = {}              # address -> buffer a graph may use
        self.on_cuda = self.device.type == "cuda"
        self._capturing = (torch._C._cuda_isCurrentStreamCapturing if self.on_cuda
                           else lambda: False)

    def get(self, nbytes: int, key=None):
        """A zero-filled buffer: of the split-K calls, or of the calls `key` names."""
        if nbytes == 0:
            return None
        if key is None:
            nbytes += QZ_WORKSPACE_COUNTERS
        buf = self.bufs.get(key)
        if buf is None or buf.numel() < nbytes or self._capturing():
            return self._other(key, nbytes, torch.zeros)
        return buf

    def get_scratch(self, nbytes: int):
        """A buffer for calls whose workspace is plain scratch (GPTQ, the W4A4
        GEMM's quantized activations): not zero-filled, and not one that other
        calls count on."""
        buf = self.bufs.get("scratch")
        if buf is None or buf.numel() < nbytes or self._capturing():
            return self._other("scratch", nbytes, torch.empty)
        return buf

    def _other(self, key, nbytes, make):
        """The buffer of a call in a capture, or of one that needs a larger one."""
        buf = self.bufs.get(key)
        fits = buf is not None and buf.numel() >= nbytes
        if self._capturing():
            if not fits:                # filled, and kept, by the graph alone
                return make(max(nbytes, 256), dtype=torch.uint8, device=self.device)
            self.captured[buf.data_ptr()] = buf
            return buf
        if buf is not None and self.on_cuda:    # calls of the current stream may still use it
            buf.record_stream(torch.cuda.current_stream(self.device))
        self.bufs[key] = make(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        return self.bufs[key]


def _ws_args(workspace, nbytes, device, key=None):
    """Pointer and size of the call's workspace (`key`: see Workspace.get).
    Called inside ``torch.cuda.stream(launch stream)``: a temporary workspace
    is then allocated and zero-filled on the stream the kernel runs on, so the
    fill is ordered before the kernel and the caching allocator hands the
    memory out again only to work queued after it on that stream."""
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
    elif isinstance(workspace, Workspace):
        buf = workspace.get(nbytes, key)
        if not workspace.on_cuda:
            raise ValueError("the workspace must live on a CUDA device")
        return buf.data_ptr(), buf.numel()
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def qz_quantize_pack(w, bits=4, symmetric=False, group_size=128, codes=None, scales=None,
                     zeros=None, workspace=None, stream=None):
    """Quantize an N x K bf16 matrix; returns (codes uint8, scales bf16, zeros uint8 | None)."""
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("w must be a 2-D bf16 tensor")
    N, K = w.shape
    qz_packed_bytes(N, K, bits, symmetric, group_size)      # validates the format
    dev = w.device
    st = _launch_stream(stream, dev)
    with _on(stream):
        if codes is None:
            codes = torch.empty((N, K // 2) if bits == 4 else (N, K), dtype=torch.uint8,
                                device=dev)
        if scales is None:
            shape = (1,) if group_size == 0 else (N, K // group_size)
            scales = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        if zeros is None and not symmetric:
            shape = (1,) if group_size == 0 else (N, K // group_size)
            zeros = torch.empty(shape, dtype=torch.uint8, device=dev)
        ws_ptr, ws_bytes = _ws_args(workspace, qz_workspace_bytes(QZ_OP_QUANTIZE_PACK, 1, N, K,
                                                                  group_size), dev, "quantize")
        _check(lib.qz_quantize_pack(_ptr(w), N, K, bits, int(symmetric), group_size,
                                    _ptr(codes), _ptr(scales),
                                    _ptr(zeros) if not symmetric else None, ws_ptr, ws_bytes,
                                    _handle(st)), "qz_quantize_pack")
    return codes, scales, (None if symmetric else zeros)


def qz_dequantize(codes, scales, zeros, N, K, bits=4, symmetric=False, group_size=128,
                  out=None, stream=None):
    """w_hat = bf16(S * (q - Z)) as an N x K bf16 tensor."""
    dev = codes.device
    st = _launch_stream(stream, dev)
    with _on(stream):
        if out is None:
            out = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
        _check(lib.qz_dequantize(_ptr(codes), _ptr(scales), _ptr(zeros), N, K, bits,
                                 int(symmetric), group_size, _ptr(out), _handle(st)),
               "qz_dequantize")
    return out


def _matmul_out(a, N, y):
    if a.dtype != torch.bfloat16 or a.dim() != 2:
        raise ValueError("a must be a 2-D bf16 tensor")
    if y is None:
        y = torch.empty((a.shape[0], N), dtype=torch.bfloat16, device=a.device)
    return y


def qz_w4a16_gemv(a, codes, scales, zeros, N, K, group_size=128, y=None, workspace=None,
                  stream=None):
    """y = a * w_hat^T for int4 asymmetric group-wise weights, M <= 16."""
    st = _launch_stream(stream, a.device)
    M = a.shape[0]
    with _on(stream):
        y = _matmul_out(a, N, y)
        nbytes = qz_workspace_bytes(QZ_OP_W4A16_GEMV, M, N, K, group_size)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, a.device)
        _check(lib.qz_w4a16_gemv(_ptr(a), _ptr(codes), _ptr(scales), _ptr(zeros), M, N, K,
                                 group_size, _ptr(y), ws_ptr, ws_bytes, _handle(st)),
               "qz_w4a16_gemv")
    return y


def qz_w4a16_gemm(a, codes, scales, zeros, N, K, group_size=128, y=None, workspace=None,
                  stream=None):
    """y = a * w_hat^T for int4 asymmetric group-wise weights, any M."""
    st = _launch_stream(stream, a.device)
    M = a.shape[0]
    with _on(stream):
        y = _matmul_out(a, N, y)
        nbytes = qz_workspace_bytes(QZ_OP_W4A16_GEMM, M, N, K, group_size)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, a.device)
        _check(lib.qz_w4a16_gemm(_ptr(a), _ptr(codes), _ptr(scales), _ptr(zeros), M, N, K,
                                 group_size, _ptr(y), ws_ptr, ws_bytes, _handle(st)),
               "qz_w4a16_gemm")
    return y


def qz_w8a16_gemv(a, codes, scales, N, K, y=None, workspace=None, stream=None):
    """y = a * w_hat^T for int8 symmetric per-channel weights, M <= 16."""
    st = _launch_stream(stream, a.device)
    M = a.shape[0]
    with _on(stream):
        y = _matmul_out(a, N, y)
        nbytes = qz_workspace_bytes(QZ_OP_W8A16_GEMV, M, N, K, K)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, a.device)
        _check(lib.qz_w8a16_gemv(_ptr(a), _ptr(codes), _ptr(scales), M, N, K, _ptr(y),
                                 ws_ptr, ws_bytes, _handle(st)), "qz_w8a16_gemv")
    return y


def qz_w8a16_gemm(a, codes, scales, N, K, y=None, workspace=None, stream=None):
    """y = a * w_hat^T for int8 symmetric per-channel weights, any M."""
    st = _launch_stream(stream, a.device)
    M = a.shape[0]
    with _on(stream):
        y = _matmul_out(a, N, y)
        nbytes = qz_workspace_bytes(QZ_OP_W8A16_GEMM, M, N, K, K)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, a.device)
        _check(lib.qz_w8a16_gemm(_ptr(a), _ptr(codes), _ptr(scales), M, N, K, _ptr(y),
                                 ws_ptr, ws_bytes, _handle(st)), "qz_w8a16_gemm")
    return y


def qz_gptq_quantize(w, x, bits=4, symmetric=False, group_size=128, damp=0.01, codes=None,
                     scales=None, zeros=None, workspace=None, stream=None):
    """GPTQ of one layer: ``w`` (N x K bf16) with calibration samples ``x``
    (n x K bf16); returns (codes, scales, zeros | None) in the packed format
    of :func:`qz_quantize_pack`."""
    if w.dtype != torch.bfloat16 or w.dim() != 2 or x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("w and x must be 2-D bf16 tensors")
    N, K = w.shape
    if x.shape[1] != K:
        raise ValueError("x must have K columns")
    qz_packed_bytes(N, K, bits, symmetric, group_size)      # validates the format
    dev = w.device
    st = _launch_stream(stream, dev)
    with _on(stream):
        if codes is None:
            codes = torch.empty((N, K // 2) if bits == 4 else (N, K), dtype=torch.uint8,
                                device=dev)
        if scales is None:
            scales = torch.empty((N, K // group_size), dtype=torch.bfloat16, device=dev)
        if zeros is None and not symmetric:
            zeros = torch.empty((N, K // group_size), dtype=torch.uint8, device=dev)
        nbytes = qz_workspace_bytes(QZ_OP_GPTQ, 1, N, K, group_size)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        elif isinstance(workspace, Workspace):
            workspace = workspace.get_scratch(nbytes)
        _check(lib.qz_gptq_quantize(_ptr(w), _ptr(x), N, K, x.shape[0], bits, int(symmetric),
                                    group_size, float(damp), _ptr(codes), _ptr(scales),
                                    _ptr(zeros) if not symmetric else None, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _handle(st)),
               "qz_gptq_quantize")
    return codes, scales, (None if symmetric else zeros)


def qz_fp4_packed_bytes(N, K, kind):
    c, s = _sz(), _sz()
    _check(lib.qz_fp4_packed_bytes(N, K, kind, ctypes.byref(c), ctypes.byref(s)),
           "qz_fp4_packed_bytes")
    return c.value, s.value


def qz_fp4_quantize(w, kind, codes=None, scales=None, tensor_scale=None, stream=None):
    """FP4 with block scales: returns (codes uint8 N x K/2, block scales uint8,
    tensor scale fp32 tensor of one element (NVFP4) or None)."""
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("w must be a 2-D bf16 tensor")
    N, K = w.shape
    qz_fp4_packed_bytes(N, K, kind)                      # validates the shape
    dev = w.device
    st = _launch_stream(stream, dev)
    with _on(stream):
        if codes is None:
            codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        if scales is None:
            scales = torch.empty((N, K // FP4_BLOCK[kind]), dtype=torch.uint8, device=dev)
        if tensor_scale is None and kind == QZ_FP4_NV:
            tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
        _check(lib.qz_fp4_quantize(_ptr(w), N, K, kind, _ptr(codes), _ptr(scales),
                                   _ptr(tensor_scale) if kind == QZ_FP4_NV else None,
                                   _handle(st)), "qz_fp4_quantize")
    return codes, scales, (tensor_scale if kind == QZ_FP4_NV else None)


def qz_fp4_dequantize(codes, scales, tensor_scale, N, K, kind, out=None, stream=None):
    """The dequantized FP4 weights as an N x K bf16 tensor."""
    dev = codes.device
    st = _launch_stream(stream, dev)
    with _on(stream):
        if out is None:
            out = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
        _check(lib.qz_fp4_dequantize(_ptr(codes), _ptr(scales), _ptr(tensor_scale), N, K, kind,
                                     _ptr(out), _handle(st)), "qz_fp4_dequantize")
    return out


def qz_fp4a16_gemv(a, codes, scales, tensor_scale, N, K, kind, y=None, workspace=None,
                   stream=None):
    """y = a * w_hat^T for FP4 weights with block scales, M <= 16."""
    st = _launch_stream(stream, a.device)
    M = a.shape[0]
    with _on(stream):
        y = _matmul_out(a, N, y)
        nbytes = qz_workspace_bytes(QZ_OP_FP4A16_GEMV, M, N, K, 0)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, a.device)
        _check(lib.qz_fp4a16_gemv(_ptr(a), _ptr(codes), _ptr(scales), _ptr(tensor_scale), M, N,
                                  K, kind, _ptr(y), ws_ptr, ws_bytes, _handle(st)),
               "qz_fp4a16_gemv")
    return y


def qz_fp4_mma_scale_bytes(rows, K, kind) -> int:
    out = _sz()
    _check(lib.qz_fp4_mma_scale_bytes(rows, K, kind, ctypes.byref(out)), "qz_fp4_mma_scale_bytes")
    return out.value


def qz_fp4_scales_to_mma(scales, rows, K, kind, out=None, stream=None):
    """Block scales as qz_fp4_quantize writes them -> the MMA scale layout
    (uint8 tensor of qz_fp4_mma_scale_bytes(rows, K, kind) bytes)."""
    st = _launch_stream(stream, scales.device)
    with _on(stream):
        if out is None:
            out = torch.empty(qz_fp4_mma_scale_bytes(rows, K, kind), dtype=torch.uint8,
                              device=scales.device)
        _check(lib.qz_fp4_scales_to_mma(_ptr(scales), rows, K, kind, _ptr(out), _handle(st)),
               "qz_fp4_scales_to_mma")
    return out


def qz_fp4a4_gemm(a, codes, scales_mma, tensor_scale, N, K, kind, y=None, workspace=None,
                  stream=None):
    """W4A4: y = a_hat * w_hat^T with the activations quantized to the same FP4
    kind inside the call.  `workspace`: a uint8 tensor, a Workspace (its
    scratch buffer is used) or None; after the call it holds the quantized
    activations."""
    st = _launch_stream(stream, a.device)
    M = a.shape[0]
    with _on(stream):
        y = _matmul_out(a, N, y)
        nbytes = qz_workspace_bytes(QZ_OP_FP4A4_GEMM, M, N, K, 0)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=a.device)
        elif isinstance(workspace, Workspace):
            workspace = workspace.get_scratch(nbytes)
        _check(lib.qz_fp4a4_gemm(_ptr(a), _ptr(codes), _ptr(scales_mma), _ptr(tensor_scale), M,
                                 N, K, kind, _ptr(y), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _handle(st)),
               "qz_fp4a4_gemm")
    return y


# ---------------------------------------------------------------------------
# low-rank adapters beside a packed projection
# ---------------------------------------------------------------------------
def _lora_args(a, N, K, lora_a, lora_b, adapters, lora_scales):
    """Addresses of the adapter arrays, adapters and rank."""
    dev = a.device
    if a.dtype is not torch.bfloat16 or a.dim() != 2 or a.shape[1] != K or not a.is_cuda:
        raise ValueError("a must be an (M, K) bf16 tensor on a CUDA device")
    if (lora_a.dtype is not torch.bfloat16 or lora_b.dtype is not torch.bfloat16 or
            lora_a.dim() != 3 or lora_b.dim() != 3):
        raise ValueError("lora_a and lora_b must be 3-D bf16 tensors")
    n, rank = lora_a.shape[0], lora_a.shape[1]
    if lora_a.shape[2] != K or lora_b.shape[0] != n or lora_b.shape[1] != N or \
            lora_b.shape[2] != rank:
        raise ValueError("lora_a must be (adapters, rank, K) and lora_b (adapters, N, rank)")
    if adapters.dtype is not torch.int32 or adapters.dim() != 1 or \
            adapters.shape[0] != a.shape[0]:
        raise ValueError("adapters must be an int32 tensor of M indices")
    if lora_scales.dtype is not torch.float32 or lora_scales.dim() != 1 or \
            lora_scales.shape[0] != n:
        raise ValueError("lora_scales must be an fp32 tensor with one value per adapter")
    for t in (a, lora_a, lora_b, adapters, lora_scales):
        if t.device != dev or not t.is_contiguous():
            raise ValueError("a and the adapter tensors must be contiguous and on one device")
    return (lora_a.data_ptr(), lora_b.data_ptr(), adapters.data_ptr(), lora_scales.data_ptr(), n,
            rank)


def _array(t, name, dtype, n, dev):
    """Address of a contiguous tensor of n values on `dev`."""
    if t.dtype is not dtype or t.numel() != n or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values on a's device")
    return t.data_ptr()


def qz_w4a16_lora_gemv(a, codes, scales, zeros, N, K, lora_a, lora_b, adapters, lora_scales,
                       group_size=128, y=None, workspace=None, stream=None):
    """y = a * w_hat^T + lora_scales[r] * (a * A_r^T) * B_r^T for int4 asymmetric
    weights, M <= 64 tokens, each with the adapter r = adapters[m] (none when
    negative).  lora_a: (adapters, rank, K), lora_b: (adapters, N, rank) bf16."""
    dev = a.device
    la, lb, ids, ls, n, rank = _lora_args(a, N, K, lora_a, lora_b, adapters, lora_scales)
    M = a.shape[0]
    if group_size < 1:
        raise ValueError("group_size must be positive")
    with _scope(dev, stream):
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        yp = _array(y, "y", torch.bfloat16, M * N, dev)
        nbytes = qz_workspace_bytes(QZ_OP_W4A16_LORA_GEMV, M, N, K, group_size)
        cp = _array(codes, "codes", torch.uint8, N * K // 2, dev)
        sp = _array(scales, "scales", torch.bfloat16, N * (K // group_size), dev)
        zp = _array(zeros, "zeros", torch.uint8, N * (K // group_size), dev)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, dev)
        _check(lib.qz_w4a16_lora_gemv(a.data_ptr(), cp, sp, zp, M, N, K, group_size, la, lb, ids, ls,
                                      n, rank, yp, ws_ptr, ws_bytes, _stream_of(dev, stream)),
               "qz_w4a16_lora_gemv")
    return y


def qz_w8a16_lora_gemv(a, codes, scales, N, K, lora_a, lora_b, adapters, lora_scales, y=None,
                       workspace=None, stream=None):
    """The same for int8 symmetric per-channel weights."""
    dev = a.device
    la, lb, ids, ls, n, rank = _lora_args(a, N, K, lora_a, lora_b, adapters, lora_scales)
    M = a.shape[0]
    with _scope(dev, stream):
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        yp = _array(y, "y", torch.bfloat16, M * N, dev)
        nbytes = qz_workspace_bytes(QZ_OP_W8A16_LORA_GEMV, M, N, K, K)
        cp = _array(codes, "codes", torch.uint8, N * K, dev)
        sp = _array(scales, "scales", torch.bfloat16, N, dev)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, dev)
        _check(lib.qz_w8a16_lora_gemv(a.data_ptr(), cp, sp, M, N, K, la, lb, ids, ls, n, rank, yp,
                                      ws_ptr, ws_bytes, _stream_of(dev, stream)),
               "qz_w8a16_lora_gemv")
    return y


# ---------------------------------------------------------------------------
# paged 4-bit key/value cache
# ---------------------------------------------------------------------------
_KV4_BYTES = {}


def qz_kv4_cache_bytes(num_pages, kv_heads, head_dim, page_size, group_size=128) -> int:
    """Bytes of a cache of `num_pages` pages of `page_size` tokens (see qz.h)."""
    key = (int(num_pages), int(kv_heads), int(head_dim), int(page_size), int(group_size))
    v = _KV4_BYTES.get(key)
    if v is None:
        b = _sz()
        _check(lib.qz_kv4_cache_bytes(*key, ctypes.byref(b)), "qz_kv4_cache_bytes")
        v = _KV4_BYTES[key] = b.value
    return v


_NO_SCOPE = contextlib.nullcontext()


class _Scope:
    """Makes `dev` (and `stream`) current for a call's allocations and launch."""

    def __init__(self, dev, stream):
        self.dev, self.stream = dev, stream

    def __enter__(self):
        self.guard = torch.cuda.device(self.dev)
        self.guard.__enter__()
        self.on = _on(self.stream)
        self.on.__enter__()

    def __exit__(self, *exc):
        self.on.__exit__(*exc)
        self.guard.__exit__(*exc)


def _scope(dev, stream):
    if stream is None and dev.index == torch.cuda.current_device():
        return _NO_SCOPE
    return _Scope(dev, stream)


# the current stream's handle without a Stream object (3 us less per call)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_of(dev, stream):
    """Handle of the stream a call runs on: `stream`, else `dev`'s current one."""
    if stream is None:
        return _current_raw_stream(torch.cuda.current_device() if dev.index is None else dev.index)
    return stream.cuda_stream


def _heads(t, name, dev):
    """Address and token stride of a (T, heads, head_dim) bf16 tensor whose
    heads and values are contiguous (tokens may lie further apart)."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.device != dev:
        raise ValueError(f"{name} must be a (tokens, heads, head_dim) bf16 tensor on the "
                         "cache's device")
    n, h, d = t.shape
    if t.is_contiguous():
        return t.data_ptr(), h * d
    st = t.stride()
    if (d > 1 and st[2] != 1) or (h > 1 and st[1] != d):
        raise ValueError(f"{name}: heads and values of a token must be contiguous")
    return t.data_ptr(), (st[0] if n > 1 else h * d)


def _kv4_args(cache, page_table, kv_lens, cu_tokens, kv_heads, head_dim, page_size, group_size):
    """Addresses of the four shared arrays, B, pages in the cache, pages per sequence."""
    dev = cache.device
    i32 = torch.int32
    if not (cache.is_cuda and cache.dtype is torch.uint8 and cache.is_contiguous()):
        raise ValueError("cache must be a contiguous uint8 tensor on a CUDA device")
    if not (page_table.dtype is i32 and kv_lens.dtype is i32 and cu_tokens.dtype is i32 and
            page_table.device == dev and kv_lens.device == dev and cu_tokens.device == dev and
            page_table.is_contiguous() and kv_lens.is_contiguous() and cu_tokens.is_contiguous()):
        raise ValueError("page_table, kv_lens and cu_tokens must be contiguous int32 tensors on "
                         "the cache's device")
    if page_table.dim() != 2 or kv_lens.dim() != 1 or cu_tokens.dim() != 1:
        raise ValueError("page_table must be 2-D, kv_lens and cu_tokens 1-D")
    B, width = page_table.shape
    if kv_lens.shape[0] != B or cu_tokens.shape[0] != B + 1:
        raise ValueError("page_table, kv_lens and cu_tokens must have B, B and B + 1 rows")
    pages = cache.numel() // qz_kv4_cache_bytes(1, kv_heads, head_dim, page_size, group_size)
    return (cache.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(), cu_tokens.data_ptr(), B,
            pages, width)


def qz_kv4_append(cache, k, v, page_table, kv_lens, cu_tokens, page_size, group_size=128,
                  stream=None):
    """Quantize new tokens' keys and values into the paged 4-bit cache.

    cache: uint8 tensor of :func:`qz_kv4_cache_bytes` bytes; k, v: (T, kv_heads,
    head_dim) bf16 (views of a fused projection are fine); page_table (B,
    max_pages), kv_lens (B) and cu_tokens (B + 1): int32 tensors.  Tokens
    cu_tokens[b]..cu_tokens[b + 1] - 1 become the last ones of sequence b, whose
    length with them is kv_lens[b].
    """
    dev = cache.device
    kp, ks = _heads(k, "k", dev)
    vp, vs = _heads(v, "v", dev)
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    T, H, D = k.shape
    c, pt, kl, cu, B, pages, width = _kv4_args(cache, page_table, kv_lens, cu_tokens, H, D,
                                               page_size, group_size)
    if T == 0:
        return
    with _scope(dev, stream):
        status = lib.qz_kv4_append(c, kp, vp, ks, vs, pt, kl, cu, T, B, H, D, page_size,
                                   group_size, pages, width, _stream_of(dev, stream))
    if status:
        raise QzError(status, "qz_kv4_append")


def qz_kv4_read(cache, page_table, kv_lens, cu_tokens, tokens, kv_heads, head_dim, page_size,
                group_size=128, k=None, v=None, stream=None):
    """The last cu_tokens[b + 1] - cu_tokens[b] cached tokens of every sequence
    as bf16: returns (k, v), each (tokens, kv_heads, head_dim)."""
    dev = cache.device
    c, pt, kl, cu, B, pages, width = _kv4_args(cache, page_table, kv_lens, cu_tokens, kv_heads,
                                               head_dim, page_size, group_size)
    shape = (tokens, kv_heads, head_dim)
    for t in (k, v):
        if t is not None and (t.dtype is not torch.bfloat16 or tuple(t.shape) != shape or
                              t.device != dev or not t.is_contiguous()):
            raise ValueError("k and v must be contiguous (tokens, kv_heads, head_dim) bf16 tensors "
                             "on the cache's device")
    with _scope(dev, stream):
        if k is None:
            k = cache.new_empty(shape, dtype=torch.bfloat16)
        if v is None:
            v = torch.empty_like(k)
        if tokens == 0:
            return k, v
        status = lib.qz_kv4_read(c, pt, kl, cu, tokens, B, kv_heads, head_dim, page_size,
                                 group_size, pages, width, k.data_ptr(), v.data_ptr(),
                                 _stream_of(dev, stream))
    if status:
        raise QzError(status, "qz_kv4_read")
    return k, v


def qz_kv4_attention(q, cache, page_table, kv_lens, cu_tokens, kv_heads, page_size,
                     group_size=128, scale=None, window=0, out=None, workspace=None, stream=None):
    """Attention of (T, q_heads, head_dim) bf16 queries over the 4-bit cache
    (causal; the queries of sequence b are its last tokens; `window` > 0 lets a
    query see its last `window` keys).  scale defaults to head_dim ** -0.5."""
    dev = cache.device
    qp, qs = _heads(q, "q", dev)
    T, H, D = q.shape
    c, pt, kl, cu, B, pages, width = _kv4_args(cache, page_table, kv_lens, cu_tokens, kv_heads, D,
                                               page_size, group_size)
    with _scope(dev, stream):
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        if T == 0:
            return out
        op, os_ = _heads(out, "out", dev)
        nbytes = qz_workspace_bytes(QZ_OP_KV4_ATTENTION, 1, 1, D, 0)
        ws_ptr, ws_bytes = _ws_args(workspace, nbytes, dev, ("kv4_attention", D))
        status = lib.qz_kv4_attention(qp, qs, c, pt, kl, cu, T, B, H, kv_heads, D, page_size,
                                      group_size, pages, width,
                                      D ** -0.5 if scale is None else scale, window, op, os_,
                                      ws_ptr, ws_bytes, _stream_of(dev, stream))
    if status:
        raise QzError(status, "qz_kv4_attention")
    return out


def qz_set_device_wait_limit(limit: int) -> None:
    lib.qz_set_device_wait_limit(int(limit))


def qz_set_launch_overlap(mode: int) -> None:
    """Launch overlap of the decode GEMV with the preceding kernel (see qz.h)."""
    _check(lib.qz_set_launch_overlap(int(mode)), "qz_set_launch_overlap")


def qz_device_status() -> int:
    return int(lib.qz_device_status())
