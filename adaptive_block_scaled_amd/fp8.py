"""8-bit floating point with a scale for each block of 128, and its matrix product:
the Python binding of include/if4_fp8.h, for the layers or steps that four bits
cost too much.

A quantized matrix is (codes, scales), both uint8: E4M3 codes [rows, K]
(`codes.view(torch.float8_e4m3fn)` are their values) and the exponents of the
blocks of 128 along K, value = code * 2^(byte - 127): [rows, ceil(K/128)], or
[ceil(rows/128), ceil(K/128)] of squares of 128 x 128, which weights have, so that
the weight and its transpose hold the same values.

The three products of a layer y = x w^T, with x [M, K] and w [N, K]:

    y  = gemm(*quantize(x), *quantize(w, square=True))
    dx = gemm(*quantize(dy), *quantize_t(w, square=True))
    dw = gemm(*quantize_t(dy), *quantize_t(x), dtype=torch.float32)

As in the rest of the binding, arguments are checked and marshalled here, all work
runs in the HIP kernels of libif4.so on torch's current stream, and nothing
records a gradient.
"""
import ctypes

import torch

from . import if4
from .if4 import _check, _dtype_code, _input, _ld, _need, _on, lib

try:
    from . import _op_call
except ImportError as e:
    raise ImportError(f"the C++ calls ({if4.HERE}/_op_call.so) do not load ({e}); build them with "
                      "`python -m adaptive_block_scaled_amd.build`") from e

EXPORTS = ("if4_fp8_quantize", "if4_fp8_quantize_t", "if4_fp8_gemm", "if4_fp8_gemm_workspace")
BLOCK = 128

# torch.cuda.current_stream(device).cuda_stream without the Stream object
_raw_stream = torch._C._cuda_getCurrentRawStream


def _declare():
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for f in (lib.if4_fp8_quantize, lib.if4_fp8_quantize_t):
        f.restype = ci
        f.argtypes = [vp, ci, i64, i64, i64, ci, vp, vp, vp]
    lib.if4_fp8_gemm.restype = ci
    lib.if4_fp8_gemm.argtypes = [vp, vp, vp, vp, ci, i64, i64, i64, vp, ci, i64, vp, i64, vp]
    lib.if4_fp8_gemm_workspace.restype = i64
    lib.if4_fp8_gemm_workspace.argtypes = [i64, i64, i64]


_declare()
_op_call.bind_fp8(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in EXPORTS))


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _quantize(fn, name, x, rows, k, square, out):
    shape = (_blocks(rows) if square else rows, _blocks(k))
    if out is None:
        codes = torch.empty((rows, k), dtype=torch.uint8, device=x.device)
        scales = torch.empty(shape, dtype=torch.uint8, device=x.device)
    else:
        codes, scales = out
        _need(codes, "codes", (rows, k), torch.uint8, x.device)
        _need(scales, "scales", shape, torch.uint8, x.device)
    st = _on(x.get_device(), fn, x.data_ptr(), _dtype_code(x.dtype), *x.shape, _ld(x), 1 if square else 0,
             codes.data_ptr(), scales.data_ptr(), _raw_stream(x.get_device()))
    _check(name, st)
    return codes, scales


def quantize(x: torch.Tensor, square: bool = False, out=None):
    """Quantize a 2-D [rows, K] CUDA tensor (fp32 or bf16, unit stride along dim 1,
    16-byte aligned rows, K a multiple of 16).  Returns (codes uint8 [rows, K], scales
    uint8 [rows, ceil(K/128)], or [ceil(rows/128), ceil(K/128)] with `square`); `out`
    may pass preallocated (codes, scales)."""
    if out is None:
        q = _op_call.quantize(x, bool(square), False)
        if type(q) is tuple:
            return q
        if q:
            _check("if4_fp8_quantize", q)
    _input(x)
    return _quantize(lib.if4_fp8_quantize, "if4_fp8_quantize", x, x.shape[0], x.shape[1], square, out)


def quantize_t(x: torch.Tensor, square: bool = False, out=None):
    """quantize(x.T) without the transposed copy, for x [K, rows], K a multiple of 16."""
    if out is None:
        q = _op_call.quantize(x, bool(square), True)
        if type(q) is tuple:
            return q
        if q:
            _check("if4_fp8_quantize_t", q)
    _input(x)
    return _quantize(lib.if4_fp8_quantize_t, "if4_fp8_quantize_t", x, x.shape[1], x.shape[0], square, out)


def workspace_bytes(m: int, n: int, k: int) -> int:
    """Bytes of workspace that gemm() takes for these sizes (0 for most)."""
    need = lib.if4_fp8_gemm_workspace(m, n, k)
    if need < 0:
        _check("if4_fp8_gemm_workspace", -need)
    return need


def gemm(a_codes, a_scales, w_codes, w_scales, dtype=torch.bfloat16, out=None, workspace=None) -> torch.Tensor:
    """C[M, N] = A[M, K] W[N, K]^T, summed in fp32, of `dtype` (bf16 or fp32; products
    enter an fp32 result whole, but for operands that bf16 does not hold, those of scale bytes
    0, 1, 2 and from 247 on; a bf16 one cut 13 bits below the largest of their 8 neighbours).
    A has blocks of one row, W blocks of one row or squares, as its scales' shape says.
    `out` may pass C with a row stride, `workspace` a uint8 tensor of workspace_bytes()."""
    if out is None and workspace is None and (dtype is torch.bfloat16 or dtype is torch.float32):
        c = _op_call.gemm(a_codes, a_scales, w_codes, w_scales, dtype is torch.bfloat16)
        if type(c) is int:
            _check("if4_fp8_gemm", c)
        elif c is not None:
            return c
    for name, t in (("a_codes", a_codes), ("w_codes", w_codes), ("w_scales", w_scales)):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D tensor")
    (m, k), n, dev = a_codes.shape, w_codes.shape[0], a_codes.device
    blocks = _blocks(k)
    square = w_scales.shape[0] != n
    _need(a_codes, "a_codes", (m, k), torch.uint8, dev)
    _need(a_scales, "a_scales", (m, blocks), torch.uint8, dev)
    _need(w_codes, "w_codes", (n, k), torch.uint8, dev)
    _need(w_scales, "w_scales", (_blocks(n) if square else n, blocks), torch.uint8, dev)
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=dev)
    else:
        _need(out, "out", (m, n), out.dtype, dev, dense=False)
    need = workspace_bytes(m, n, k)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != dev or \
                workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {dev}")
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    index = a_codes.get_device()
    st = _on(index, lib.if4_fp8_gemm, a_codes.data_ptr(), a_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(),
             1 if square else 0, m, n, k, out.data_ptr(), _dtype_code(out.dtype), _ld(out),
             workspace.data_ptr() if need else None, need, _raw_stream(index))
    _check("if4_fp8_gemm", st)
    return out
