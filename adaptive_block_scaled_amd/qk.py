"""Norms of queries and keys for each head with the position rotation in the same
pass, and its gradients: the Python binding of include/if4_qk.h, which gives the
formulas.

`norm_rotate` takes q and k as the projection leaves them (column slices of its
output are fine) and gives what attention and the cache take;
`norm_rotate_backward` gives the gradients of q, k and of both weights.
`rotation_table` makes the cosines and sines.  As in the rest of the binding, arguments
are checked and marshalled here, all work runs in the HIP kernels of libif4.so on
torch's current stream, and nothing records a gradient.
"""
import ctypes
import math

import torch

from .fp8 import _op_call
from .if4 import _check, _dtype_code, _on, lib

EXPORTS = ("if4_norm_rotate", "if4_norm_rotate_backward", "if4_norm_rotate_backward_workspace")

# torch.cuda.current_stream(device).cuda_stream without the Stream object
_raw_stream = torch._C._cuda_getCurrentRawStream


class _Part(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_stride_token", ctypes.c_int64), ("x_stride_head", ctypes.c_int64),
                ("g", ctypes.c_void_p), ("g_stride_token", ctypes.c_int64), ("g_stride_head", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("y_stride_token", ctypes.c_int64), ("y_stride_head", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("d_weight", ctypes.c_void_p), ("heads", ctypes.c_int64)]


class _Args(ctypes.Structure):
    _fields_ = [("q", _Part), ("k", _Part), ("table", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("tokens", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("rotary", ctypes.c_int64),
                ("table_rows", ctypes.c_int64), ("eps", ctypes.c_float), ("interleaved", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def _declare():
    vp, i64, ci, args = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(_Args)
    lib.if4_norm_rotate.restype = ci
    lib.if4_norm_rotate.argtypes = [args, vp]
    lib.if4_norm_rotate_backward.restype = ci
    lib.if4_norm_rotate_backward.argtypes = [args, vp, i64, vp]
    lib.if4_norm_rotate_backward_workspace.restype = i64
    lib.if4_norm_rotate_backward_workspace.argtypes = [args]


_declare()
_op_call.bind_qk(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in EXPORTS))


def rotation_table(rows: int, rotary: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of positions 0 .. rows - 1, fp32 [rows, rotary]: pair i of a
    position turns by position * base^(-2 i / rotary).  The angles are computed in 64
    bits: in 32, those of far positions are off by more than a cosine's own rounding."""
    if rotary <= 0 or rotary % 8:
        raise ValueError(f"rotary must be a positive multiple of 8, not {rotary}")
    i = torch.arange(rotary // 2, dtype=torch.float64, device=device)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * base ** (-2 * i / rotary)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _vectors(t, name, shape, dtype, device):
    """A [tokens, heads, D] tensor with unit stride along D and free others."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dim() != 3 or t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along its last dim")


def _plain(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {tuple(shape)}")


def _strides(t):
    """Strides between tokens and between heads; those that nothing is apart by are 0."""
    return tuple(s if n > 1 else 0 for n, s in zip(t.shape[:2], t.stride()))


def _written(t, name):
    """An output's vectors must not overlap: strides as of some order of tokens and heads."""
    (n, h, d), (st, sh, _) = t.shape, t.stride()
    if n > 1 and st < d or h > 1 and sh < d or n > 1 and h > 1 and st < sh * (h - 1) + d and sh < st * (n - 1) + d:
        raise ValueError(f"{name} must have vectors that do not overlap")


def _args(q, k, q_weight, k_weight, table, positions, eps, interleaved, out_dtype):
    for t, name in ((q, "q"), (k, "k")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3:
            raise ValueError(f"{name} must be a 3-D CUDA tensor [tokens, heads, D]")
    tokens, _, dim = q.shape
    dev = q.device
    _vectors(q, "q", q.shape, q.dtype, dev)
    _vectors(k, "k", (tokens, k.shape[1], dim), q.dtype, dev)
    _plain(q_weight, "q_weight", (dim,), torch.float32, dev)
    _plain(k_weight, "k_weight", (dim,), torch.float32, dev)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D tensor [positions, rotary]")
    _plain(table, "table", table.shape, torch.float32, dev)
    _plain(positions, "positions", (tokens,), torch.int64, dev)
    eps = float(eps)
    if not 0 <= eps < math.inf:
        raise ValueError("eps must be finite and not negative")
    a = _Args(table=table.data_ptr(), positions=positions.data_ptr(), tokens=tokens, head_dim=dim,
              rotary=table.shape[1], table_rows=table.shape[0], eps=eps, interleaved=1 if interleaved else 0,
              dtype=_dtype_code(q.dtype), out_dtype=_dtype_code(out_dtype))
    for part, x, w in ((a.q, q, q_weight), (a.k, k, k_weight)):
        part.x, part.weight, part.heads = x.data_ptr(), w.data_ptr(), x.shape[1]
        part.x_stride_token, part.x_stride_head = _strides(x)
    return a, dev


def _results(a, shapes, dtype, dev, out):
    if out is None:
        out = tuple(torch.empty(shape, dtype=dtype, device=dev) for shape in shapes)
    else:
        out = tuple(out)
        for t, name, shape in zip(out, "qk", shapes):
            _vectors(t, f"out's {name}", shape, dtype, dev)
            _written(t, f"out's {name}")
    for part, y in zip((a.q, a.k), out):
        part.y = y.data_ptr()
        part.y_stride_token, part.y_stride_head = _strides(y)
    return out


def norm_rotate(q, k, q_weight, k_weight, table, positions, *, eps: float = 1e-6, interleaved: bool = False,
                dtype=None, out=None):
    """q [tokens, heads, D] and k [tokens, kv_heads, D] (fp32 or bf16, unit stride along
    D, other strides multiples of 16 bytes), each vector divided by the root of its mean
    square, times its weight (fp32 [D]), and its first table.shape[1] values rotated by the
    token's position (int64 [tokens]): pairs (i, i + rotary/2), or (2i, 2i + 1) where
    `interleaved`.  D is a multiple of 8 up to 256, rotary one of 16 (interleaved: 8) up to D.

    Returns (q, k) of `dtype` (default: q's); `out` may pass them, q itself for q and k itself
    for k among others, but nothing that overlaps an input otherwise.  A token whose position is outside the table is skipped: its outputs keep
    what they hold, and are unset without `out`."""
    if out is None and (dtype is None or dtype is torch.bfloat16 or dtype is torch.float32):
        bf16 = (dtype or getattr(q, "dtype", None)) is torch.bfloat16
        y = _op_call.norm_rotate(q, k, q_weight, k_weight, table, positions, eps, interleaved, bf16)
        if type(y) is tuple:
            return y
        if y:
            _check("if4_norm_rotate", y)
    if dtype is None:
        dtype = q.dtype if out is None and isinstance(q, torch.Tensor) else out[0].dtype
    a, dev = _args(q, k, q_weight, k_weight, table, positions, eps, interleaved, dtype)
    out = _results(a, (q.shape, k.shape), dtype, dev, out)
    st = _on(q.get_device(), lib.if4_norm_rotate, a, _raw_stream(q.get_device()))
    _check("if4_norm_rotate", st)
    return out


def workspace_bytes(head_dim: int) -> int:
    """Bytes of workspace that norm_rotate_backward() takes."""
    need = lib.if4_norm_rotate_backward_workspace(_Args(head_dim=head_dim))
    if need < 0:
        _check("if4_norm_rotate_backward_workspace", -need)
    return need


def norm_rotate_backward(dq, dk, q, k, q_weight, k_weight, table, positions, *, eps: float = 1e-6,
                         interleaved: bool = False, out=None, workspace=None):
    """Gradients of norm_rotate(q, k, ...) for the gradients dq and dk of its outputs (fp32
    or bf16, both alike).  Returns (q's, k's, q_weight's, k_weight's): the first two of q's
    dtype (`out` may pass them), the weights' fp32 [D].  Skipped tokens have zero gradients
    and add nothing.  `workspace` may pass a uint8 tensor of workspace_bytes()."""
    if out is None and workspace is None:
        grads = _op_call.norm_rotate_backward(dq, dk, q, k, q_weight, k_weight, table, positions, eps, interleaved)
        if type(grads) is tuple:
            return grads
        if grads:
            _check("if4_norm_rotate_backward", grads)
    if not isinstance(dq, torch.Tensor):
        raise ValueError("dq must be a 3-D CUDA tensor [tokens, heads, D]")
    a, dev = _args(q, k, q_weight, k_weight, table, positions, eps, interleaved, dq.dtype)
    for part, g, x, name in ((a.q, dq, q, "dq"), (a.k, dk, k, "dk")):
        _vectors(g, name, x.shape, dq.dtype, dev)
        part.g = g.data_ptr()
        part.g_stride_token, part.g_stride_head = _strides(g)
    dx = _results(a, (q.shape, k.shape), q.dtype, dev, out)
    need = lib.if4_norm_rotate_backward_workspace(a)
    if need < 0:
        _check("if4_norm_rotate_backward", -need)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != dev or workspace.dtype != torch.uint8 or \
            not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {dev}")
    dw = torch.empty(2, q.shape[2], dtype=torch.float32, device=dev)
    for part, row in ((a.q, dw[0]), (a.k, dw[1])):
        part.d_weight = row.data_ptr()
        if part.heads == 0:
            row.zero_()
    st = _on(q.get_device(), lib.if4_norm_rotate_backward, a, workspace.data_ptr(), need, _raw_stream(q.get_device()))
    _check("if4_norm_rotate_backward", st)
    return (*dx, dw[0], dw[1])
