"""memra-gb300: Q8_0 decode GEMV / verify GEMM / routed-expert GEMV for GB300.

A thin Python binding over the C ABI in ``include/memra.h`` (``libmemra.so``).
The binding only marshals arguments: it checks tensor devices, dtypes, shapes and
contiguity, allocates outputs with torch when the caller passes none, and calls the
library on the current torch CUDA stream.  Every step of the computation runs in the
library's sm_103a kernels; there is no fallback.  If the library has not been built
(``block_quantized_decode_quantize_gb300.build.build()``) loading it raises.

The decode step's other half is here too: the page plan of a step (memra_kv_plan), a paged
KV cache in 8 bits (memra_kv_append_q8, memra_kv_read_q8), attention over it
(memra_kv_attention_q8) and the routing to experts (memra_moe_route).

Tensor conventions (all on one CUDA device, contiguous):
  wq  int8 [N, K]          Q8_0 quants            wd  float16 [N, K/32]  Q8_0 scales
  xq  int8 [M, K]          q8_1 quants            xd  float32 [M, K/32]  q8_1 scales
  y   float32 [M, N]       (the GEMV takes and returns 1-D x / y)
"""
import ctypes
import importlib.util
import os
import warnings

import torch

from . import build as _build

MEMRA_OK = 0
MEMRA_BF16 = 0
MEMRA_F32 = 1
MAX_M = 16
MAX_TOP_K = 64
MOE_NOALLOC_SCRATCH_FLOATS = 65536
KV_ATTENTION_WORKSPACE_BYTES = 33554432

_STATUS = {0: "MEMRA_OK", 1: "MEMRA_ERR_INVALID_ARG", 2: "MEMRA_ERR_ALIGNMENT",
           3: "MEMRA_ERR_UNSUPPORTED", 4: "MEMRA_ERR_CUDA"}


class MemraError(RuntimeError):
    def __init__(self, fn, status, cuda_error=0):
        self.status = status
        self.cuda_error = cuda_error
        msg = "%s returned %s" % (fn, _STATUS.get(status, status))
        if cuda_error:
            msg += " (cudaError %d)" % cuda_error
        super().__init__(msg)


_lib = None

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32

_SIGS = {
    "memra_quantize_q8_0": [_p, _i64, _i64, _p, _p, _p],
    "memra_quantize_q8_1": [_p, _i32, _i64, _i64, _p, _p, _p],
    "memra_q8_0_gemv": [_p, _p, _i64, _i64, _p, _p, _p, _p],
    "memra_quantize_q4_0": [_p, _i64, _i64, _p, _p, _p],
    "memra_repack_q8_0": [_p, _i64, _i64, _p, _p, _p],
    "memra_quantize_nvfp4": [_p, _i64, _i64, _p, _p, _p, _p],
    "memra_read_stream": [_p, _i64, _p, _i32, _p],
    "memra_nvfp4_gemm_small_m": [_p, _p, ctypes.c_float, _i64, _i64, _i64, _p, _p, _p, _p],
    "memra_nvfp4_gemv": [_p, _p, ctypes.c_float, _i64, _i64, _p, _p, _p, _p],
    "memra_nvfp4_moe_gemv": [_p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _p, _i32, _p, _p,
                             _p],
    "memra_nvfp4_moe_gemv_tokens": [_p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _p, _p,
                                    _i32, _p, _p, _p, _p],
    "memra_repack_q4_0": [_p, _i64, _i64, _p, _p, _p],
    "memra_q4_0_gemv": [_p, _p, _i64, _i64, _p, _p, _p, _p],
    "memra_q4_0_gemm_small_m": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p],
    "memra_q4_0_moe_gemv": [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _p, _i32, _p, _p, _p],
    "memra_q8_0_gemm_small_m": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p],
    "memra_q8_0_gemm_small_m_mma": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p],
    "memra_q8_0_quant_gemm": [_p, _p, _i64, _i64, _i64, _p, _i32, _p, _p],
    "memra_q8_0_moe_gemv": [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _p, _i32, _p, _p, _p],
    "memra_q8_0_moe_gemv_tokens": [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _p, _p, _i32,
                                   _p, _p, _p, _p],
    "memra_q4_0_moe_gemv_tokens": [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _p, _p, _i32,
                                   _p, _p, _p, _p],
    "memra_q8_0_moe_ffn_tokens": [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _p, _i32,
                                  _p, _p, _p, _p],
    "memra_q4_0_moe_ffn": [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _i32, _p, _p, _p,
                           _p],
    "memra_nvfp4_moe_ffn": [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _i32, _p,
                            _p, _p, _p],
    "memra_q4_0_moe_ffn_tokens": [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _p, _i32,
                                  _p, _p, _p, _p],
    "memra_nvfp4_moe_ffn_tokens": [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64,
                                   _p, _i32, _p, _p, _p, _p],
    "memra_swiglu_quantize_q8_1": [_p, _i64, _i64, _p, _p, _p],
    "memra_q8_0_moe_ffn": [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _i32, _p, _p, _p,
                           _p],
    "memra_q8_0_moe_ffn_noalloc": [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _i32, _p,
                                   _p, _p],
    "memra_q8_0_block_dots": [_p, _i64, _i64, _p, _i64, _p, _p],
    "memra_debug_set_wait_test": [_i64, _i64],
    "memra_kv_plan": [_p, _p, _i64, _i64, _p, _i64, _p, _p, _i64, _i64, _p, _p, _p, _p, _p, _p,
                      _p],
    "memra_kv_append_q8": [_p, _p, _i32, _i64, _i64, _i64, _p, _p, _p, _p, _p, _i64, _i64, _i64,
                           _i64, _i64, _p, _p],
    "memra_kv_read_q8": [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _i64, _i32, _p, _p, _p,
                         _p],
    "memra_kv_attention_q8": [_p, _i32, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _i64, _i64, _i64,
                              _i64, _i64, _p, _i64, _i64, _p, _p, ctypes.c_float, _i64, _p, _p,
                              _p, _p, _p],
    "memra_moe_route": [_p, _i32, _i64, _i64, _i64, _p, _i32, _i64, _i64, _i64, _i64, _i32,
                        ctypes.c_float, _p, _p, _p],
}


def library_path():
    return _build.LIB


def lib():
    """The loaded C library (ctypes), with argument types set for every entry point."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError("libmemra.so is not built (expected at %s); run "
                               "block_quantized_decode_quantize_gb300.build.build()" % path)
        L = ctypes.CDLL(path)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.memra_status_string.argtypes = [ctypes.c_int]
        L.memra_status_string.restype = ctypes.c_char_p
        L.memra_last_cuda_error.restype = ctypes.c_int32
        L.memra_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(name, status):
    if status != MEMRA_OK:
        L = lib()
        raise MemraError(name, status, L.memra_last_cuda_error() if status == 4 else 0)


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, name, dtype, device=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def memra_quantize_q8_0(w, wq=None, wd=None):
    """fp32 weights [N, K] -> (wq int8 [N, K], wd float16 [N, K/32])."""
    _need(w, "w", torch.float32)
    N, K = w.shape
    if wq is None:
        wq = torch.empty((N, K), dtype=torch.int8, device=w.device)
    if wd is None:
        wd = torch.empty((N, K // 32), dtype=torch.float16, device=w.device)
    _need(wq, "wq", torch.int8, w.device, (N, K))
    _need(wd, "wd", torch.float16, w.device, (N, K // 32))
    with torch.cuda.device(w.device):
        _check("memra_quantize_q8_0",
               lib().memra_quantize_q8_0(_ptr(w), N, K, _ptr(wq), _ptr(wd), _stream(w)))
    return wq, wd


def memra_quantize_q4_0(w, wq4=None, wd=None):
    """fp32 weights [N, K] -> (wq4 uint8 [N, K/2] packed 4-bit codes, wd float16 [N, K/32])."""
    _need(w, "w", torch.float32)
    N, K = w.shape
    if wq4 is None:
        wq4 = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    if wd is None:
        wd = torch.empty((N, K // 32), dtype=torch.float16, device=w.device)
    _need(wq4, "wq4", torch.uint8, w.device, (N, K // 2))
    _need(wd, "wd", torch.float16, w.device, (N, K // 32))
    with torch.cuda.device(w.device):
        _check("memra_quantize_q4_0",
               lib().memra_quantize_q4_0(_ptr(w), N, K, _ptr(wq4), _ptr(wd), _stream(w)))
    return wq4, wd


def _blocks(blocks, N, K, block_bytes):
    _need(blocks, "blocks", torch.uint8)
    if K % 32 != 0 or blocks.numel() != N * (K // 32) * block_bytes:
        raise ValueError("blocks must hold N * K/32 blocks of %d bytes (N=%d, K=%d), got %d bytes"
                         % (block_bytes, N, K, blocks.numel()))


def memra_repack_q8_0(blocks, N, K, wq=None, wd=None):
    """GGUF Q8_0 block bytes (uint8, N * K/32 * 34) -> (wq int8 [N, K], wd float16 [N, K/32])."""
    _blocks(blocks, N, K, 34)
    if wq is None:
        wq = torch.empty((N, K), dtype=torch.int8, device=blocks.device)
    if wd is None:
        wd = torch.empty((N, K // 32), dtype=torch.float16, device=blocks.device)
    _need(wq, "wq", torch.int8, blocks.device, (N, K))
    _need(wd, "wd", torch.float16, blocks.device, (N, K // 32))
    with torch.cuda.device(blocks.device):
        _check("memra_repack_q8_0",
               lib().memra_repack_q8_0(_ptr(blocks), N, K, _ptr(wq), _ptr(wd), _stream(blocks)))
    return wq, wd


def memra_repack_q4_0(blocks, N, K, wq4=None, wd=None):
    """GGUF Q4_0 block bytes (uint8, N * K/32 * 18) -> (wq4 uint8 [N, K/2], wd float16 [N, K/32])."""
    _blocks(blocks, N, K, 18)
    if wq4 is None:
        wq4 = torch.empty((N, K // 2), dtype=torch.uint8, device=blocks.device)
    if wd is None:
        wd = torch.empty((N, K // 32), dtype=torch.float16, device=blocks.device)
    _need(wq4, "wq4", torch.uint8, blocks.device, (N, K // 2))
    _need(wd, "wd", torch.float16, blocks.device, (N, K // 32))
    with torch.cuda.device(blocks.device):
        _check("memra_repack_q4_0",
               lib().memra_repack_q4_0(_ptr(blocks), N, K, _ptr(wq4), _ptr(wd), _stream(blocks)))
    return wq4, wd


def memra_read_stream(buf, sink=None, ctas_per_sm=2):
    """Read every byte of the CUDA tensor `buf` once (diagnostic read stream); returns the
    per-CTA xor sink (uint32, zeroed here when not given)."""
    if not isinstance(buf, torch.Tensor) or not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    nbytes = buf.numel() * buf.element_size()
    if sink is None:
        sms = torch.cuda.get_device_properties(buf.device).multi_processor_count
        sink = torch.zeros((sms * ctas_per_sm,), dtype=torch.int32, device=buf.device)
    with torch.cuda.device(buf.device):
        _check("memra_read_stream",
               lib().memra_read_stream(_ptr(buf), nbytes, _ptr(sink), ctas_per_sm,
                                       _stream(buf)))
    return sink


def memra_quantize_q8_1(x, xq=None, xd=None):
    """Activations [M, K] (bf16 or fp32) -> (xq int8 [M, K], xd float32 [M, K/32])."""
    if x.dtype == torch.bfloat16:
        dt = MEMRA_BF16
    elif x.dtype == torch.float32:
        dt = MEMRA_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    _need(x, "x", x.dtype)
    M, K = x.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if xd is None:
        xd = torch.empty((M, K // 32), dtype=torch.float32, device=x.device)
    _need(xq, "xq", torch.int8, x.device, (M, K))
    _need(xd, "xd", torch.float32, x.device, (M, K // 32))
    with torch.cuda.device(x.device):
        _check("memra_quantize_q8_1",
               lib().memra_quantize_q8_1(_ptr(x), dt, M, K, _ptr(xq), _ptr(xd), _stream(x)))
    return xq, xd


def memra_q8_0_gemm_small_m(wq, wd, xq, xd, y=None):
    """y [M, N] = W (Q8_0) x (q8_1) for M <= 16 activation rows (two weight passes above 8)."""
    _need(wq, "wq", torch.int8)
    N, K = wq.shape
    dev = wq.device
    _need(wd, "wd", torch.float16, dev, (N, K // 32))
    _need(xq, "xq", torch.int8, dev)
    M = xq.shape[0]
    _need(xq, "xq", torch.int8, dev, (M, K))
    _need(xd, "xd", torch.float32, dev, (M, K // 32))
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (M, N))
    with torch.cuda.device(dev):
        _check("memra_q8_0_gemm_small_m",
               lib().memra_q8_0_gemm_small_m(_ptr(wq), _ptr(wd), N, K, M, _ptr(xq), _ptr(xd),
                                             _ptr(y), _stream(wq)))
    return y


def memra_q8_0_gemm_small_m_mma(wq, wd, xq, xd, y=None):
    """memra_q8_0_gemm_small_m with the block sums on the tensor cores (bit-identical
    results; K a multiple of 1024 up to 5120, N >= 16)."""
    _need(wq, "wq", torch.int8)
    N, K = wq.shape
    dev = wq.device
    _need(wd, "wd", torch.float16, dev, (N, K // 32))
    _need(xq, "xq", torch.int8, dev)
    M = xq.shape[0]
    _need(xq, "xq", torch.int8, dev, (M, K))
    _need(xd, "xd", torch.float32, dev, (M, K // 32))
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (M, N))
    with torch.cuda.device(dev):
        _check("memra_q8_0_gemm_small_m_mma",
               lib().memra_q8_0_gemm_small_m_mma(_ptr(wq), _ptr(wd), N, K, M, _ptr(xq),
                                                 _ptr(xd), _ptr(y), _stream(wq)))
    return y


def memra_q8_0_quant_gemm(wq, wd, x, y=None):
    """y [M, N] = W (Q8_0) x, with x [M, K] (bf16 or fp32) quantised to q8_1 inside the
    kernel; bit-identical to memra_quantize_q8_1 followed by memra_q8_0_gemm_small_m."""
    _need(wq, "wq", torch.int8)
    N, K = wq.shape
    dev = wq.device
    _need(wd, "wd", torch.float16, dev, (N, K // 32))
    if x.dtype == torch.bfloat16:
        dt = MEMRA_BF16
    elif x.dtype == torch.float32:
        dt = MEMRA_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    _need(x, "x", x.dtype, dev)
    M = x.shape[0]
    _need(x, "x", x.dtype, dev, (M, K))
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (M, N))
    with torch.cuda.device(dev):
        _check("memra_q8_0_quant_gemm",
               lib().memra_q8_0_quant_gemm(_ptr(wq), _ptr(wd), N, K, M, _ptr(x), dt, _ptr(y),
                                           _stream(wq)))
    return y


def memra_q8_0_gemv(wq, wd, xq, xd, y=None):
    """y [N] = W (Q8_0) x (q8_1) for one activation row (xq [K], xd [K/32])."""
    _need(wq, "wq", torch.int8)
    N, K = wq.shape
    dev = wq.device
    _need(wd, "wd", torch.float16, dev, (N, K // 32))
    _need(xq, "xq", torch.int8, dev, (K,))
    _need(xd, "xd", torch.float32, dev, (K // 32,))
    if y is None:
        y = torch.empty((N,), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (N,))
    with torch.cuda.device(dev):
        _check("memra_q8_0_gemv",
               lib().memra_q8_0_gemv(_ptr(wq), _ptr(wd), N, K, _ptr(xq), _ptr(xd), _ptr(y),
                                     _stream(wq)))
    return y


def memra_q4_0_gemm_small_m(wq4, wd, xq, xd, y=None):
    """y [M, N] = W (Q4_0: wq4 uint8 [N, K/2], wd float16 [N, K/32]) x (q8_1), M <= 16."""
    _need(wq4, "wq4", torch.uint8)
    N, K2 = wq4.shape
    K = 2 * K2
    dev = wq4.device
    _need(wd, "wd", torch.float16, dev, (N, K // 32))
    _need(xq, "xq", torch.int8, dev)
    M = xq.shape[0]
    _need(xq, "xq", torch.int8, dev, (M, K))
    _need(xd, "xd", torch.float32, dev, (M, K // 32))
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (M, N))
    with torch.cuda.device(dev):
        _check("memra_q4_0_gemm_small_m",
               lib().memra_q4_0_gemm_small_m(_ptr(wq4), _ptr(wd), N, K, M, _ptr(xq), _ptr(xd),
                                             _ptr(y), _stream(wq4)))
    return y


def memra_quantize_nvfp4(w, codes=None, scales=None, g=None):
    """fp32 weights [N, K] -> (codes uint8 [N, K/2], scales uint8 E4M3 bits [N, K/16],
    g float32 [1] on the device: the tensor scale)."""
    _need(w, "w", torch.float32)
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty((N, K // 16), dtype=torch.uint8, device=w.device)
    if g is None:
        g = torch.empty((1,), dtype=torch.float32, device=w.device)
    _need(codes, "codes", torch.uint8, w.device, (N, K // 2))
    _need(scales, "scales", torch.uint8, w.device, (N, K // 16))
    _need(g, "g", torch.float32, w.device, (1,))
    with torch.cuda.device(w.device):
        _check("memra_quantize_nvfp4",
               lib().memra_quantize_nvfp4(_ptr(w), N, K, _ptr(codes), _ptr(scales), _ptr(g),
                                          _stream(w)))
    return codes, scales, g


def memra_nvfp4_gemm_small_m(codes, scales, g, xq, xd, y=None):
    """y [M, N] = W (NVFP4: codes uint8 [N, K/2], scales uint8 E4M3 [N, K/16], tensor
    scale g, a Python float) x (q8_1), M <= 16."""
    _need(codes, "codes", torch.uint8)
    N, K2 = codes.shape
    K = 2 * K2
    dev = codes.device
    _need(scales, "scales", torch.uint8, dev, (N, K // 16))
    _need(xq, "xq", torch.int8, dev)
    M = xq.shape[0]
    _need(xq, "xq", torch.int8, dev, (M, K))
    _need(xd, "xd", torch.float32, dev, (M, K // 32))
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (M, N))
    with torch.cuda.device(dev):
        _check("memra_nvfp4_gemm_small_m",
               lib().memra_nvfp4_gemm_small_m(_ptr(codes), _ptr(scales), float(g), N, K, M,
                                              _ptr(xq), _ptr(xd), _ptr(y), _stream(codes)))
    return y


def memra_nvfp4_gemv(codes, scales, g, xq, xd, y=None):
    """y [N] = W (NVFP4) x (q8_1) for one activation row (xq [K], xd [K/32])."""
    _need(codes, "codes", torch.uint8)
    N, K2 = codes.shape
    K = 2 * K2
    dev = codes.device
    _need(scales, "scales", torch.uint8, dev, (N, K // 16))
    _need(xq, "xq", torch.int8, dev, (K,))
    _need(xd, "xd", torch.float32, dev, (K // 32,))
    if y is None:
        y = torch.empty((N,), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (N,))
    with torch.cuda.device(dev):
        _check("memra_nvfp4_gemv",
               lib().memra_nvfp4_gemv(_ptr(codes), _ptr(scales), float(g), N, K, _ptr(xq),
                                      _ptr(xd), _ptr(y), _stream(codes)))
    return y


def memra_q4_0_gemv(wq4, wd, xq, xd, y=None):
    """y [N] = W (Q4_0) x (q8_1) for one activation row (xq [K], xd [K/32])."""
    _need(wq4, "wq4", torch.uint8)
    N, K2 = wq4.shape
    K = 2 * K2
    dev = wq4.device
    _need(wd, "wd", torch.float16, dev, (N, K // 32))
    _need(xq, "xq", torch.int8, dev, (K,))
    _need(xd, "xd", torch.float32, dev, (K // 32,))
    if y is None:
        y = torch.empty((N,), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (N,))
    with torch.cuda.device(dev):
        _check("memra_q4_0_gemv",
               lib().memra_q4_0_gemv(_ptr(wq4), _ptr(wd), N, K, _ptr(xq), _ptr(xd), _ptr(y),
                                     _stream(wq4)))
    return y


def _moe_gemv(fn, wq_bank, qdtype, kmul, wd_bank, ids, gate_w, xq, xd, x_per_expert, y,
              dev_status):
    _need(wq_bank, "wq_bank", qdtype)
    E, N, Kq = wq_bank.shape
    K = Kq * kmul
    dev = wq_bank.device
    _need(wd_bank, "wd_bank", torch.float16, dev, (E, N, K // 32))
    _need(ids, "ids", torch.int32, dev)
    top_k = ids.shape[0]
    if gate_w is not None:
        _need(gate_w, "gate_w", torch.float32, dev, (top_k,))
    xpe = 1 if x_per_expert else 0
    if xpe:
        _need(xq, "xq", torch.int8, dev, (top_k, K))
        _need(xd, "xd", torch.float32, dev, (top_k, K // 32))
    else:
        _need(xq, "xq", torch.int8, dev, (K,))
        _need(xd, "xd", torch.float32, dev, (K // 32,))
    yshape = (N,) if gate_w is not None else (top_k, N)
    if y is None:
        y = torch.empty(yshape, dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, yshape)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    with torch.cuda.device(dev):
        _check(fn, getattr(lib(), fn)(_ptr(wq_bank), _ptr(wd_bank), E, N, K, _ptr(ids),
                                      _ptr(gate_w), top_k, _ptr(xq), _ptr(xd), xpe, _ptr(y),
                                      _ptr(dev_status), _stream(wq_bank)))
    return y


def memra_q8_0_moe_gemv(wq_bank, wd_bank, ids, gate_w, xq, xd, x_per_expert, y=None,
                        dev_status=None):
    """Routed-expert GEMV.  wq_bank int8 [E, N, K], wd_bank float16 [E, N, K/32],
    ids int32 [top_k], gate_w float32 [top_k] or None.  x_per_expert=False: xq [K],
    xd [K/32]; True: xq [top_k, K], xd [top_k, K/32].  Returns y [top_k, N] without
    gate weights, [N] with them."""
    return _moe_gemv("memra_q8_0_moe_gemv", wq_bank, torch.int8, 1, wd_bank, ids, gate_w, xq,
                     xd, x_per_expert, y, dev_status)


def memra_q4_0_moe_gemv(wq4_bank, wd_bank, ids, gate_w, xq, xd, x_per_expert, y=None,
                        dev_status=None):
    """memra_q8_0_moe_gemv on a Q4_0 bank: wq4_bank uint8 [E, N, K/2] (packed codes),
    wd_bank float16 [E, N, K/32]."""
    return _moe_gemv("memra_q4_0_moe_gemv", wq4_bank, torch.uint8, 2, wd_bank, ids, gate_w, xq,
                     xd, x_per_expert, y, dev_status)


def _moe_gemv_tokens(fn, wq_bank, qdtype, kmul, wd_bank, ids, gate_w, xq, xd, x_per_expert,
                     y, workspace, dev_status):
    _need(wq_bank, "wq_bank", qdtype)
    E, N, Kq = wq_bank.shape
    K = Kq * kmul
    dev = wq_bank.device
    _need(wd_bank, "wd_bank", torch.float16, dev, (E, N, K // 32))
    _need(ids, "ids", torch.int32, dev)
    T, top_k = ids.shape
    if gate_w is not None:
        _need(gate_w, "gate_w", torch.float32, dev, (T, top_k))
    xpe = 1 if x_per_expert else 0
    rows = (T, top_k) if xpe else (T,)
    _need(xq, "xq", torch.int8, dev, rows + (K,))
    _need(xd, "xd", torch.float32, dev, rows + (K // 32,))
    yshape = (T, N) if gate_w is not None else (T, top_k, N)
    if y is None:
        y = torch.empty(yshape, dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, yshape)
    if gate_w is not None:
        if workspace is None:
            workspace = torch.empty((T, top_k, N), dtype=torch.float32, device=dev)
        _need(workspace, "workspace", torch.float32, dev, (T, top_k, N))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    with torch.cuda.device(dev):
        _check(fn, getattr(lib(), fn)(_ptr(wq_bank), _ptr(wd_bank), E, N, K, _ptr(ids),
                                      _ptr(gate_w), T, top_k, _ptr(xq), _ptr(xd), xpe, _ptr(y),
                                      _ptr(workspace), _ptr(dev_status), _stream(wq_bank)))
    return y


def memra_q8_0_moe_gemv_tokens(wq_bank, wd_bank, ids, gate_w, xq, xd, x_per_expert, y=None,
                               workspace=None, dev_status=None):
    """Routed experts for a batch of tokens.  ids int32 [T, top_k], gate_w float32
    [T, top_k] or None.  x_per_expert=False: xq [T, K], xd [T, K/32]; True: xq
    [T, top_k, K], xd [T, top_k, K/32].  Returns y [T, top_k, N] without gate weights,
    [T, N] with them (`workspace` float32 [T, top_k, N] then holds the per-pair rows)."""
    return _moe_gemv_tokens("memra_q8_0_moe_gemv_tokens", wq_bank, torch.int8, 1, wd_bank, ids,
                            gate_w, xq, xd, x_per_expert, y, workspace, dev_status)


def memra_q4_0_moe_gemv_tokens(wq4_bank, wd_bank, ids, gate_w, xq, xd, x_per_expert, y=None,
                               workspace=None, dev_status=None):
    """memra_q8_0_moe_gemv_tokens on a Q4_0 bank (wq4_bank uint8 [E, N, K/2])."""
    return _moe_gemv_tokens("memra_q4_0_moe_gemv_tokens", wq4_bank, torch.uint8, 2, wd_bank,
                            ids, gate_w, xq, xd, x_per_expert, y, workspace, dev_status)


def memra_q8_0_moe_ffn_tokens(gu_q, gu_d, dn_q, dn_d, ids, gate_w, x, y=None, workspace=None,
                              dev_status=None):
    """memra_q8_0_moe_ffn for a batch: ids int32 [T, top_k], gate_w float32 [T, top_k],
    x [T, H] (bf16 or fp32).  Returns y float32 [T, H].  `workspace` float32
    [T * top_k * (2F + H)] holds the pairs' gate|up rows, then their down rows."""
    _need(gu_q, "gu_q", torch.int8)
    E, F2, H = gu_q.shape
    F = F2 // 2
    dev = gu_q.device
    _need(gu_d, "gu_d", torch.float16, dev, (E, F2, H // 32))
    _need(dn_q, "dn_q", torch.int8, dev, (E, H, F))
    _need(dn_d, "dn_d", torch.float16, dev, (E, H, F // 32))
    _need(ids, "ids", torch.int32, dev)
    T, top_k = ids.shape
    _need(gate_w, "gate_w", torch.float32, dev, (T, top_k))
    if x.dtype == torch.bfloat16:
        dt = MEMRA_BF16
    elif x.dtype == torch.float32:
        dt = MEMRA_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    _need(x, "x", x.dtype, dev, (T, H))
    if y is None:
        y = torch.empty((T, H), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (T, H))
    ws = T * top_k * (F2 + H)
    if workspace is None:
        workspace = torch.empty((ws,), dtype=torch.float32, device=dev)
    _need(workspace, "workspace", torch.float32, dev, (ws,))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    with torch.cuda.device(dev):
        _check("memra_q8_0_moe_ffn_tokens",
               lib().memra_q8_0_moe_ffn_tokens(_ptr(gu_q), _ptr(gu_d), _ptr(dn_q), _ptr(dn_d), E,
                                               H, F, _ptr(ids), _ptr(gate_w), T, top_k, _ptr(x),
                                               dt, _ptr(y), _ptr(workspace), _ptr(dev_status),
                                               _stream(gu_q)))
    return y


def memra_nvfp4_moe_gemv(codes_bank, scales_bank, gexp, ids, gate_w, xq, xd, x_per_expert,
                         y=None, dev_status=None):
    """Routed experts on an NVFP4 bank: codes_bank uint8 [E, N, K/2], scales_bank uint8
    E4M3 [E, N, K/16], gexp float32 [E] (each expert's tensor scale, on the device);
    the rest as memra_q8_0_moe_gemv."""
    _need(codes_bank, "codes_bank", torch.uint8)
    E, N, K2 = codes_bank.shape
    K = 2 * K2
    dev = codes_bank.device
    _need(scales_bank, "scales_bank", torch.uint8, dev, (E, N, K // 16))
    _need(gexp, "gexp", torch.float32, dev, (E,))
    _need(ids, "ids", torch.int32, dev)
    top_k = ids.shape[0]
    if gate_w is not None:
        _need(gate_w, "gate_w", torch.float32, dev, (top_k,))
    xpe = 1 if x_per_expert else 0
    rows = (top_k,) if xpe else ()
    _need(xq, "xq", torch.int8, dev, rows + (K,))
    _need(xd, "xd", torch.float32, dev, rows + (K // 32,))
    yshape = (N,) if gate_w is not None else (top_k, N)
    if y is None:
        y = torch.empty(yshape, dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, yshape)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    with torch.cuda.device(dev):
        _check("memra_nvfp4_moe_gemv",
               lib().memra_nvfp4_moe_gemv(_ptr(codes_bank), _ptr(scales_bank), _ptr(gexp), E, N,
                                          K, _ptr(ids), _ptr(gate_w), top_k, _ptr(xq), _ptr(xd),
                                          xpe, _ptr(y), _ptr(dev_status), _stream(codes_bank)))
    return y


def memra_nvfp4_moe_gemv_tokens(codes_bank, scales_bank, gexp, ids, gate_w, xq, xd,
                                x_per_expert, y=None, workspace=None, dev_status=None):
    """memra_q8_0_moe_gemv_tokens on an NVFP4 bank (layout as memra_nvfp4_moe_gemv)."""
    _need(codes_bank, "codes_bank", torch.uint8)
    E, N, K2 = codes_bank.shape
    K = 2 * K2
    dev = codes_bank.device
    _need(scales_bank, "scales_bank", torch.uint8, dev, (E, N, K // 16))
    _need(gexp, "gexp", torch.float32, dev, (E,))
    _need(ids, "ids", torch.int32, dev)
    T, top_k = ids.shape
    if gate_w is not None:
        _need(gate_w, "gate_w", torch.float32, dev, (T, top_k))
    xpe = 1 if x_per_expert else 0
    rows = (T, top_k) if xpe else (T,)
    _need(xq, "xq", torch.int8, dev, rows + (K,))
    _need(xd, "xd", torch.float32, dev, rows + (K // 32,))
    yshape = (T, N) if gate_w is not None else (T, top_k, N)
    if y is None:
        y = torch.empty(yshape, dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, yshape)
    if gate_w is not None:
        if workspace is None:
            workspace = torch.empty((T, top_k, N), dtype=torch.float32, device=dev)
        _need(workspace, "workspace", torch.float32, dev, (T, top_k, N))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    with torch.cuda.device(dev):
        _check("memra_nvfp4_moe_gemv_tokens",
               lib().memra_nvfp4_moe_gemv_tokens(_ptr(codes_bank), _ptr(scales_bank), _ptr(gexp),
                                                 E, N, K, _ptr(ids), _ptr(gate_w), T, top_k,
                                                 _ptr(xq), _ptr(xd), xpe, _ptr(y),
                                                 _ptr(workspace), _ptr(dev_status),
                                                 _stream(codes_bank)))
    return y


def memra_q8_0_moe_ffn(gu_q, gu_d, dn_q, dn_d, ids, gate_w, x, y=None, workspace=None,
                       dev_status=None):
    """One routed-expert FFN layer: gu_q int8 [E, 2F, H], gu_d float16 [E, 2F, H/32],
    dn_q int8 [E, H, F], dn_d float16 [E, H, F/32], ids int32 [top_k], gate_w float32
    [top_k], x [H] (bf16 or fp32).  Returns y float32 [H].  `workspace` (float32
    [top_k, 2F]) receives the gate|up outputs; allocated here when not given."""
    _need(gu_q, "gu_q", torch.int8)
    E, F2, H = gu_q.shape
    F = F2 // 2
    dev = gu_q.device
    _need(gu_d, "gu_d", torch.float16, dev, (E, F2, H // 32))
    _need(dn_q, "dn_q", torch.int8, dev, (E, H, F))
    _need(dn_d, "dn_d", torch.float16, dev, (E, H, F // 32))
    _need(ids, "ids", torch.int32, dev)
    top_k = ids.shape[0]
    _need(gate_w, "gate_w", torch.float32, dev, (top_k,))
    if x.dtype == torch.bfloat16:
        dt = MEMRA_BF16
    elif x.dtype == torch.float32:
        dt = MEMRA_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    _need(x, "x", x.dtype, dev, (H,))
    if y is None:
        y = torch.empty((H,), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, (H,))
    if workspace is None:
        workspace = torch.empty((top_k, F2), dtype=torch.float32, device=dev)
    _need(workspace, "workspace", torch.float32, dev, (top_k, F2))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    with torch.cuda.device(dev):
        _check("memra_q8_0_moe_ffn",
               lib().memra_q8_0_moe_ffn(_ptr(gu_q), _ptr(gu_d), _ptr(dn_q), _ptr(dn_d), E, H, F,
                                        _ptr(ids), _ptr(gate_w), top_k, _ptr(x), dt, _ptr(y),
                                        _ptr(workspace), _ptr(dev_status), _stream(gu_q)))
    return y


def _moe_ffn_4bit(fmt, gu, gu_s, gu_g, dn, dn_s, dn_g, ids, gate_w, x, y, workspace,
                  dev_status):
    """Shared marshalling of the Q4_0 and NVFP4 routed FFN entry points (one token when
    ids is 1-D, a batch of tokens when it is [T, top_k])."""
    _need(gu, "gate|up bank", torch.uint8)
    E, F2, H2 = gu.shape
    H, F = 2 * H2, F2 // 2
    dev = gu.device
    sdt, sdiv = (torch.float16, 32) if fmt == "q4_0" else (torch.uint8, 16)
    _need(gu_s, "gate|up scales", sdt, dev, (E, F2, H // sdiv))
    _need(dn, "down bank", torch.uint8, dev, (E, H, F // 2))
    _need(dn_s, "down scales", sdt, dev, (E, H, F // sdiv))
    if fmt == "nvfp4":
        _need(gu_g, "gu_g", torch.float32, dev, (E,))
        _need(dn_g, "dn_g", torch.float32, dev, (E,))
    _need(ids, "ids", torch.int32, dev)
    tokens = ids.dim() == 2
    T, top_k = (ids.shape if tokens else (1, ids.shape[0]))
    _need(gate_w, "gate_w", torch.float32, dev, tuple(ids.shape))
    if x.dtype == torch.bfloat16:
        dt = MEMRA_BF16
    elif x.dtype == torch.float32:
        dt = MEMRA_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    yshape = (T, H) if tokens else (H,)
    _need(x, "x", x.dtype, dev, yshape)
    if y is None:
        y = torch.empty(yshape, dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, dev, yshape)
    ws = T * top_k * (F2 + H) if tokens else top_k * F2
    if workspace is None:
        workspace = torch.empty((ws,), dtype=torch.float32, device=dev)
    _need(workspace, "workspace", torch.float32, dev)
    if workspace.numel() != ws:
        raise ValueError("workspace must hold %d floats" % ws)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    L = lib()
    name = "memra_%s_moe_ffn%s" % (fmt, "_tokens" if tokens else "")
    banks = ([_ptr(gu), _ptr(gu_s), _ptr(dn), _ptr(dn_s)] if fmt == "q4_0" else
             [_ptr(gu), _ptr(gu_s), _ptr(gu_g), _ptr(dn), _ptr(dn_s), _ptr(dn_g)])
    sizes = [E, H, F, _ptr(ids), _ptr(gate_w)] + ([T, top_k] if tokens else [top_k])
    with torch.cuda.device(dev):
        _check(name, getattr(L, name)(*banks, *sizes, _ptr(x), dt, _ptr(y), _ptr(workspace),
                                      _ptr(dev_status), _stream(gu)))
    return y


def memra_q4_0_moe_ffn(gu_q4, gu_d, dn_q4, dn_d, ids, gate_w, x, y=None, workspace=None,
                       dev_status=None):
    """The routed FFN layer on Q4_0 banks (gu_q4 uint8 [E, 2F, H/2], gu_d float16
    [E, 2F, H/32], dn_q4 uint8 [E, H, F/2], dn_d float16 [E, H, F/32]).  ids [top_k] for
    one token (x [H]) or [T, top_k] for a batch (x [T, H], the batched entry point)."""
    return _moe_ffn_4bit("q4_0", gu_q4, gu_d, None, dn_q4, dn_d, None, ids, gate_w, x, y,
                         workspace, dev_status)


def memra_nvfp4_moe_ffn(gu_codes, gu_scales, gu_g, dn_codes, dn_scales, dn_g, ids, gate_w, x,
                        y=None, workspace=None, dev_status=None):
    """The routed FFN layer on NVFP4 banks (codes uint8 [E, rows, K/2], E4M3 scales uint8
    [E, rows, K/16], per-expert tensor scales float32 [E] for each bank).  ids [top_k]
    for one token or [T, top_k] for a batch."""
    return _moe_ffn_4bit("nvfp4", gu_codes, gu_scales, gu_g, dn_codes, dn_scales, dn_g, ids,
                         gate_w, x, y, workspace, dev_status)


def memra_q8_0_moe_ffn_noalloc(gu_q, gu_d, dn_q, dn_d, ids, gate_w, x, y, dev_status=None):
    """memra_q8_0_moe_ffn with the gate|up workspace inside the library: the C call
    allocates no device memory (the caller provides y).  For callers that cannot
    allocate at call time; top_k * 2F must not exceed MOE_NOALLOC_SCRATCH_FLOATS.
    The first call on a device should come before any stream capture; calls that
    overlap on the GPU share one scratch array and race."""
    _need(gu_q, "gu_q", torch.int8)
    E, F2, H = gu_q.shape
    F = F2 // 2
    dev = gu_q.device
    _need(gu_d, "gu_d", torch.float16, dev, (E, F2, H // 32))
    _need(dn_q, "dn_q", torch.int8, dev, (E, H, F))
    _need(dn_d, "dn_d", torch.float16, dev, (E, H, F // 32))
    _need(ids, "ids", torch.int32, dev)
    top_k = ids.shape[0]
    _need(gate_w, "gate_w", torch.float32, dev, (top_k,))
    if x.dtype == torch.bfloat16:
        dt = MEMRA_BF16
    elif x.dtype == torch.float32:
        dt = MEMRA_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    _need(x, "x", x.dtype, dev, (H,))
    _need(y, "y", torch.float32, dev, (H,))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev, (1,))
    with torch.cuda.device(dev):
        _check("memra_q8_0_moe_ffn_noalloc",
               lib().memra_q8_0_moe_ffn_noalloc(_ptr(gu_q), _ptr(gu_d), _ptr(dn_q), _ptr(dn_d), E,
                                                H, F, _ptr(ids), _ptr(gate_w), top_k, _ptr(x),
                                                dt, _ptr(y), _ptr(dev_status), _stream(gu_q)))
    return y


def memra_swiglu_quantize_q8_1(gu, hq=None, hd=None):
    """gu float32 [R, 2F] (gate | up) -> (hq int8 [R, F], hd float32 [R, F/32])."""
    _need(gu, "gu", torch.float32)
    R, F2 = gu.shape
    F = F2 // 2
    if hq is None:
        hq = torch.empty((R, F), dtype=torch.int8, device=gu.device)
    if hd is None:
        hd = torch.empty((R, F // 32), dtype=torch.float32, device=gu.device)
    _need(hq, "hq", torch.int8, gu.device, (R, F))
    _need(hd, "hd", torch.float32, gu.device, (R, F // 32))
    with torch.cuda.device(gu.device):
        _check("memra_swiglu_quantize_q8_1",
               lib().memra_swiglu_quantize_q8_1(_ptr(gu), R, F, _ptr(hq), _ptr(hd),
                                                _stream(gu)))
    return hq, hd


def memra_q8_0_block_dots(wq, xq, s=None):
    """Exact int32 block sums s [M, N, K/32]."""
    _need(wq, "wq", torch.int8)
    N, K = wq.shape
    dev = wq.device
    _need(xq, "xq", torch.int8, dev)
    M = xq.shape[0]
    _need(xq, "xq", torch.int8, dev, (M, K))
    if s is None:
        s = torch.empty((M, N, K // 32), dtype=torch.int32, device=dev)
    _need(s, "s", torch.int32, dev, (M, N, K // 32))
    with torch.cuda.device(dev):
        _check("memra_q8_0_block_dots",
               lib().memra_q8_0_block_dots(_ptr(wq), N, K, _ptr(xq), M, _ptr(s), _stream(wq)))
    return s


# The entry points below run many times a decode step on small data, where the time of the
# call itself counts.  Each goes through the extension module _memra_binding first
# (csrc/binding.cpp), which makes the same checks in C++ and calls the same C entry point;
# where that finds anything unusual it returns None, and the long way here names the error
# or handles the case.

_fast = None


class _NoBinding:
    """Where the extension module could not be built: every call takes the long way."""

    @staticmethod
    def plan(*args):
        return None

    append = read = attention = route = plan


def _binding():
    """The extension module with the quick paths (built and loaded with the library)."""
    global _fast
    if _fast is None:
        lib()
        path = _build.BINDING
        if os.path.exists(path):
            spec = importlib.util.spec_from_file_location("_memra_binding", path)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
        else:
            mod = _NoBinding
            warnings.warn("%s is not built: calls of the cache, attention and routing take 14 to 40 us on the "
                          "host instead of 5 to 9; see block_quantized_decode_quantize_gb300.build.build()" % path,
                          RuntimeWarning, stacklevel=3)
        _fast = mod
    return _fast


def _ok(t, name, dtype, dev, shape):
    """_need for a contiguous tensor on CUDA device number `dev`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, torch.device("cuda", dev), shape)


def _rows(t, name, dev, ndim):
    """dtype code of a bf16 / fp32 tensor whose last dimension is dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is torch.bfloat16:
        dt = MEMRA_BF16
    elif t.dtype is torch.float32:
        dt = MEMRA_F32
    else:
        raise TypeError("%s must be bfloat16 or float32" % name)
    if t.get_device() != dev or dev < 0:
        raise ValueError("%s must be a CUDA tensor on the other arguments' device" % name)
    if t.dim() != ndim:
        raise ValueError("%s must have %d dimensions, got %d" % (name, ndim, t.dim()))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the last dimension of %s must be dense" % name)
    return dt


def _strides(t):
    """Strides of rows and heads of [rows, heads, D]; those of a single row or head, which
    reach nothing and may be any number, as if dense."""
    rows, heads, D = t.shape
    return (t.stride(0) if rows > 1 else heads * D), (t.stride(1) if heads > 1 else D)


# The current stream's handle without a Stream object around it (1 us less).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(name, dev, *args):
    fn = getattr(_lib if _lib is not None else lib(), name)
    stream = _raw_stream(dev)
    if torch.cuda.current_device() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        _check(name, st)


def _addr(t):
    return t.data_ptr() if t is not None else None


def _cache(kq, kd, vq, vd):
    """(device, n_pages, Hkv, page, D, block) of a cache's planes."""
    if not isinstance(kq, torch.Tensor) or kq.dim() != 4 or not isinstance(kd, torch.Tensor) \
            or kd.dim() != 3:
        raise ValueError("the cache is kq, vq [pages, Hkv, page, D] and kd, vd [pages, Hkv, "
                         "page / block]")
    dev = kq.get_device()
    n_pages, Hkv, page, D = shape = kq.shape
    blocks = kd.shape[2]
    if blocks < 1 or page % blocks:
        raise ValueError("a page of %d tokens does not hold %d scale blocks" % (page, blocks))
    if dev < 0:
        raise ValueError("kq must be a CUDA tensor")
    scales = (n_pages, Hkv, blocks)
    _ok(kq, "kq", torch.int8, dev, shape)
    _ok(vq, "vq", torch.int8, dev, shape)
    _ok(kd, "kd", torch.float32, dev, scales)
    _ok(vd, "vd", torch.float32, dev, scales)
    return dev, n_pages, Hkv, page, D, page // blocks


def memra_kv_plan(ctx_lens, new_lens, page_size, free_pages, block_table, num_tokens,
                  free_head=None, kv_lens=None, cu_q=None, slots=None, positions=None,
                  free_head_out=None, dev_status=None):
    """The page plan of one step.  ctx_lens, new_lens int32 [B] (tokens in the cache, tokens
    of this step), free_pages int32 [F], block_table int32 [B, max_pages] (its new entries
    are written in place), free_head int32 [1] or None (start of the unused free pages).
    Returns kv_lens [B], cu_q [B+1], slots [num_tokens], positions [num_tokens] and
    free_head_out [1], all int32.  free_head_out may be free_head, and kv_lens ctx_lens or
    new_lens, to advance them in place."""
    if kv_lens is None and cu_q is None and slots is None and positions is None:
        done = (_fast or _binding()).plan(ctx_lens, new_lens, page_size, free_pages, block_table,
                                          num_tokens, free_head, free_head_out, dev_status)
        if done is not None:
            return done
    if not isinstance(ctx_lens, torch.Tensor) or not ctx_lens.is_cuda or ctx_lens.dim() != 1:
        raise ValueError("ctx_lens must be a 1-D CUDA tensor")
    dev, B, T = ctx_lens.get_device(), ctx_lens.shape[0], int(num_tokens)
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    i32 = torch.int32
    _ok(ctx_lens, "ctx_lens", i32, dev, (B,))
    _ok(new_lens, "new_lens", i32, dev, (B,))
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a 1-D tensor")
    _ok(free_pages, "free_pages", i32, dev, free_pages.shape)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a 2-D tensor")
    max_pages = block_table.shape[1]
    _ok(block_table, "block_table", i32, dev, (B, max_pages))
    if free_head is not None:
        _ok(free_head, "free_head", i32, dev, (1,))
    if kv_lens is None and cu_q is None and slots is None and positions is None \
            and free_head_out is None:
        # one allocation; slots and positions first, which keeps them 16-byte aligned
        pad = -T % 4
        buf = torch.empty(2 * (T + pad) + 2 * B + 2, dtype=i32, device=ctx_lens.device)
        slots, _, positions, _, kv_lens, cu_q, free_head_out = buf.split_with_sizes(
            (T, pad, T, pad, B, B + 1, 1))
    else:
        if kv_lens is None:
            kv_lens = torch.empty((B,), dtype=i32, device=ctx_lens.device)
        if cu_q is None:
            cu_q = torch.empty((B + 1,), dtype=i32, device=ctx_lens.device)
        if slots is None:
            slots = torch.empty((T,), dtype=i32, device=ctx_lens.device)
        if positions is None:
            positions = torch.empty((T,), dtype=i32, device=ctx_lens.device)
        if free_head_out is None:
            free_head_out = torch.empty((1,), dtype=i32, device=ctx_lens.device)
        _ok(kv_lens, "kv_lens", i32, dev, (B,))
        _ok(cu_q, "cu_q", i32, dev, (B + 1,))
        _ok(slots, "slots", i32, dev, (T,))
        _ok(positions, "positions", i32, dev, (T,))
        _ok(free_head_out, "free_head_out", i32, dev, (1,))
    if dev_status is not None:
        _ok(dev_status, "dev_status", i32, dev, (1,))
    _launch("memra_kv_plan", dev, ctx_lens.data_ptr(), new_lens.data_ptr(), B, page_size,
            free_pages.data_ptr(), free_pages.shape[0], _addr(free_head), block_table.data_ptr(),
            max_pages, T, kv_lens.data_ptr(), cu_q.data_ptr(), slots.data_ptr(),
            positions.data_ptr(), free_head_out.data_ptr(), _addr(dev_status))
    return kv_lens, cu_q, slots, positions, free_head_out


def memra_kv_append_q8(k, v, slots, kq, kd, vq, vd, dev_status=None):
    """Write tokens into the cache: k, v [T, Hkv, D] (bf16 or fp32; any equal strides of 16
    bytes' multiples with the last dimension dense, so columns of a fused projection's rows
    will do), slots int32 [T] (-1: left out).  kq, vq int8 [pages, Hkv, page, D] and kd, vd
    float32 [pages, Hkv, page / block] are updated in place."""
    if (_fast or _binding()).append(k, v, slots, kq, kd, vq, vd, dev_status):
        return
    dev, n_pages, Hkv, page, D, block = _cache(kq, kd, vq, vd)
    dt = _rows(k, "k", dev, 3)
    T = k.shape[0]
    if k.shape[1] != Hkv or k.shape[2] != D:
        raise ValueError("k has shape %s, expected %s" % (tuple(k.shape), (T, Hkv, D)))
    if _rows(v, "v", dev, 3) != dt or v.shape != k.shape or _strides(v) != _strides(k):
        raise ValueError("v must have k's dtype, shape and strides")
    _ok(slots, "slots", torch.int32, dev, (T,))
    if dev_status is not None:
        _ok(dev_status, "dev_status", torch.int32, dev, (1,))
    stride_t, stride_h = _strides(k)
    _launch("memra_kv_append_q8", dev, k.data_ptr(), v.data_ptr(), dt, T, stride_t, stride_h,
            slots.data_ptr(), kq.data_ptr(), kd.data_ptr(), vq.data_ptr(), vd.data_ptr(), n_pages,
            Hkv, page, D, block, _addr(dev_status))


def memra_kv_read_q8(slots, kq, kd, vq, vd, dtype=torch.bfloat16, k=None, v=None,
                     dev_status=None):
    """Read cached tokens back as values: slots int32 [N] -> k, v [N, Hkv, D] of `dtype`
    (bfloat16 or float32); zeros where a slot is -1."""
    if k is None and v is None and (dtype is torch.bfloat16 or dtype is torch.float32):
        done = (_fast or _binding()).read(slots, kq, kd, vq, vd, dtype is torch.bfloat16,
                                          dev_status)
        if done is not None:
            return done
    dev, n_pages, Hkv, page, D, block = _cache(kq, kd, vq, vd)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D tensor")
    N = slots.shape[0]
    _ok(slots, "slots", torch.int32, dev, (N,))
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("dtype must be bfloat16 or float32")
    if k is None and v is None:
        k, v = torch.empty((2, N, Hkv, D), dtype=dtype, device=kq.device).unbind(0)
    else:
        if k is None:
            k = torch.empty((N, Hkv, D), dtype=dtype, device=kq.device)
        if v is None:
            v = torch.empty((N, Hkv, D), dtype=dtype, device=kq.device)
        _ok(k, "k", dtype, dev, (N, Hkv, D))
        _ok(v, "v", dtype, dev, (N, Hkv, D))
    if dev_status is not None:
        _ok(dev_status, "dev_status", torch.int32, dev, (1,))
    _launch("memra_kv_read_q8", dev, slots.data_ptr(), N, kq.data_ptr(), kd.data_ptr(),
            vq.data_ptr(), vd.data_ptr(), n_pages, Hkv, page, D, block,
            MEMRA_BF16 if dtype is torch.bfloat16 else MEMRA_F32, k.data_ptr(), v.data_ptr(),
            _addr(dev_status))
    return k, v


def memra_kv_attention_q8(q, kq, kd, vq, vd, block_table, kv_lens, cu_q, scale=None, window=0,
                          out=None, lse=None, workspace=None, dev_status=None):
    """Causal attention of a step's queries over the cache.  q [T, Hq, D] (bf16 or fp32,
    strided as for memra_kv_append_q8), rows cu_q[b] .. cu_q[b+1] the last tokens of
    request b's kv_lens[b]; block_table int32 [B, max_pages], kv_lens int32 [B], cu_q int32
    [B+1] (as memra_kv_plan gives them); scale defaults to D ** -0.5; window > 0 hides keys
    `window` and more before the query.  Returns out [T, Hq, D] (q's dtype) and lse float32
    [T, Hq].  `workspace` (uint8, KV_ATTENTION_WORKSPACE_BYTES, zeroed once before its first
    use) should be kept from call to call, one a stream; without one a call takes and clears
    its own."""
    if out is None and lse is None and workspace is not None and scale is not None:
        done = (_fast or _binding()).attention(q, kq, kd, vq, vd, block_table, kv_lens, cu_q,
                                               scale, window, workspace, dev_status)
        if done is not None:
            return done
    dev, n_pages, Hkv, page, D, block = _cache(kq, kd, vq, vd)
    dt = _rows(q, "q", dev, 3)
    T, Hq, qD = q.shape
    if qD != D or Hq < 1 or Hq % Hkv:
        raise ValueError("q has shape %s, expected [T, a multiple of %d, %d]"
                         % (tuple(q.shape), Hkv, D))
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a 2-D tensor")
    B, max_pages = block_table.shape
    i32 = torch.int32
    _ok(block_table, "block_table", i32, dev, (B, max_pages))
    _ok(kv_lens, "kv_lens", i32, dev, (B,))
    _ok(cu_q, "cu_q", i32, dev, (B + 1,))
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
    else:
        _ok(out, "out", q.dtype, dev, (T, Hq, D))
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    else:
        _ok(lse, "lse", torch.float32, dev, (T, Hq))
    if workspace is None:
        workspace = torch.zeros(KV_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device=q.device)
    elif workspace.numel() < KV_ATTENTION_WORKSPACE_BYTES:
        raise ValueError("workspace must hold %d bytes" % KV_ATTENTION_WORKSPACE_BYTES)
    else:
        _ok(workspace, "workspace", torch.uint8, dev, workspace.shape)
    if dev_status is not None:
        _ok(dev_status, "dev_status", i32, dev, (1,))
    stride_t, stride_h = _strides(q)
    _launch("memra_kv_attention_q8", dev, q.data_ptr(), dt, T, Hq, stride_t, stride_h,
            kq.data_ptr(), kd.data_ptr(), vq.data_ptr(), vd.data_ptr(), n_pages, Hkv, page, D,
            block, block_table.data_ptr(), B, max_pages, kv_lens.data_ptr(), cu_q.data_ptr(),
            D ** -0.5 if scale is None else scale, window, out.data_ptr(), lse.data_ptr(),
            workspace.data_ptr(), _addr(dev_status))
    return out, lse


_SCORES = {"softmax": 0, "sigmoid": 1}


def memra_moe_route(logits, top_k, bias=None, score="softmax", n_groups=1, topk_groups=1,
                    group_top=1, renormalize=True, scale=1.0, ids=None, gate_w=None):
    """Routing: logits [T, E] (bf16 or fp32, the last dimension dense) -> ids int32 [T,
    top_k] (descending rank, ties to the lowest index) and gate_w float32 [T, top_k], as the
    routed products take them.  score "softmax" or "sigmoid"; bias float32 [E] is added for
    the ranking only; with n_groups > 1 only the topk_groups best groups stay, a group
    ranked by its group_top (1 or 2) best experts' sum."""
    if ids is None and gate_w is None:
        done = (_fast or _binding()).route(logits, top_k, bias, _SCORES.get(score, -1), n_groups,
                                           topk_groups, group_top, renormalize, scale)
        if done is not None:
            return done
    dev = logits.get_device() if isinstance(logits, torch.Tensor) else -1
    dt = _rows(logits, "logits", dev, 2)
    T, E = logits.shape
    if score not in _SCORES:
        raise ValueError("score must be softmax or sigmoid, got %r" % (score,))
    if bias is not None:
        _ok(bias, "bias", torch.float32, dev, (E,))
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    else:
        _ok(ids, "ids", torch.int32, dev, (T, top_k))
    if gate_w is None:
        gate_w = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    else:
        _ok(gate_w, "gate_w", torch.float32, dev, (T, top_k))
    _launch("memra_moe_route", dev, logits.data_ptr(), dt, T, E, logits.stride(0), _addr(bias),
            _SCORES[score], n_groups, topk_groups, group_top, top_k, 1 if renormalize else 0,
            scale, ids.data_ptr(), gate_w.data_ptr())
    return ids, gate_w


def memra_debug_set_wait_test(wait_limit_cycles=0, stall_after_stages=-1):
    """Test hook: later product launches give up waiting after wait_limit_cycles SM
    cycles and, with stall_after_stages >= 0, stall after that many stages per CTA, so
    that their abort path runs (NaN outputs, status bit 2).  Defaults switch it off."""
    _check("memra_debug_set_wait_test",
           lib().memra_debug_set_wait_test(int(wait_limit_cycles), int(stall_after_stages)))


def version():
    return lib().memra_version().decode()
