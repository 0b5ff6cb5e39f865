"""Paged KV cache in IF4 and the attention that reads it: the Python binding of
include/if4_kv.h.

A cache is four uint8 tensors (KVCache): `pages` pages of `page_size` tokens,
K and V quantized to IF4 in groups of 16 along the head dimension, 4.5 bits
per value.  `append` quantizes new tokens into slots (page * page_size +
offset), `read` gives slots back as bf16 or fp32, `attention` attends from the
newest tokens of a batch of sequences, each with its row of a page table.

As in the rest of the binding, arguments are checked and marshalled here and
all work runs in the HIP kernels of libif4.so, on torch's current stream.  A
call whose arguments are in order is marshalled in C++ (csrc/kv_call.cpp: 3 to
5 us less than here, of calls that take 5 to 10); what that turns down comes to
the checks below, which say what is wrong.

These are operators of serving: none records a gradient, whatever its inputs
require (as the rest of the binding does not).
"""
import ctypes
import math
from typing import NamedTuple

import torch

from . import if4
from .if4 import GROUP, MODE_ADAPTIVE, _check, _dtype_code, _need, lib

try:
    from . import _kv_call
except ImportError as e:
    raise ImportError(f"the KV cache's C++ calls ({if4.HERE}/_kv_call.so) do not load ({e}); build them "
                      "with `python -m adaptive_block_scaled_amd.build`") from e

EXPORTS = ("if4_kv_append", "if4_kv_read", "if4_kv_attention", "if4_kv_attention_workspace",
           "if4_kv_attention_workspace_most")
HEAD_DIMS = (64, 128, 256)


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("k_exp", ctypes.c_int32), ("v_exp", ctypes.c_int32)]


class _Attention(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("out_stride_token", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("seq_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("total_q", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("max_q", ctypes.c_int64), ("max_len", ctypes.c_int64),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32)]


# torch.cuda.current_stream(device).cuda_stream without the Stream object
_raw_stream = torch._C._cuda_getCurrentRawStream


def _declare():
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    cache, args = ctypes.POINTER(_Cache), ctypes.POINTER(_Attention)
    lib.if4_kv_append.restype = ci
    lib.if4_kv_append.argtypes = [cache, vp, vp, ci, i64, i64, i64, i64, i64, vp, ci, vp]
    lib.if4_kv_read.restype = ci
    lib.if4_kv_read.argtypes = [cache, vp, i64, vp, vp, ci, vp]
    lib.if4_kv_attention.restype = ci
    lib.if4_kv_attention.argtypes = [cache, args, vp, i64, vp]
    for f in (lib.if4_kv_attention_workspace, lib.if4_kv_attention_workspace_most):
        f.restype = i64
        f.argtypes = [cache, args]


_declare()
_kv_call.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in EXPORTS[:4]))


class KVCache(NamedTuple):
    """The tensors of a cache (uint8, contiguous; layouts in include/if4_kv.h)."""
    k_codes: torch.Tensor   # [pages, kv_heads, page_size, D/2]
    k_scales: torch.Tensor  # [pages, kv_heads, page_size, D/16]
    v_codes: torch.Tensor   # [pages, kv_heads, page_size/16, 16, 16, D/32]
    v_scales: torch.Tensor  # [pages, kv_heads, page_size/16, D/16, 16]


def empty(pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda") -> KVCache:
    """A cache of zeros (every slot reads as zeros)."""
    _sizes(page_size, kv_heads, head_dim)
    return KVCache(*(torch.zeros(shape, dtype=torch.uint8, device=device)
                     for shape in _shapes(pages, page_size, kv_heads, head_dim)))


def _sizes(page_size, kv_heads, head_dim):
    if head_dim not in HEAD_DIMS:
        raise ValueError(f"head_dim must be one of {HEAD_DIMS}, not {head_dim}")
    if page_size <= 0 or page_size % 16:
        raise ValueError(f"page_size must be a multiple of 16, not {page_size}")
    if kv_heads <= 0:
        raise ValueError(f"kv_heads must be positive, not {kv_heads}")


def _shapes(pages, page_size, kv_heads, head_dim):
    tiles = page_size // 16
    return ((pages, kv_heads, page_size, head_dim // 2),
            (pages, kv_heads, page_size, head_dim // GROUP),
            (pages, kv_heads, tiles, 16, 16, head_dim // 32),
            (pages, kv_heads, tiles, head_dim // GROUP, 16))


def _held(v, bits):
    """The int nearest to v that a C integer of `bits` bits holds.  ctypes takes the
    low bits of a larger one, which can name a value in order; the nearest one
    means the same to a size or a bound, and is refused where v has to be."""
    top = 1 << (bits - 1)
    return max(-top, min(int(v), top - 1))


def _is(t, shape, dtype, index) -> bool:
    """Whether t is a contiguous tensor of this shape and type on CUDA device
    `index`: the check of a call that is in order.  It costs a third of a
    microsecond; only one that fails goes on to _need, which says what is
    wrong."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and
            t.shape == shape and t.is_contiguous())


def _cache(cache: KVCache, k_exp: int, v_exp: int):
    kc, ks, vc, vs = cache
    if not isinstance(kc, torch.Tensor) or not kc.is_cuda or kc.dim() != 4:
        raise ValueError("k_codes must be a CUDA tensor [pages, kv_heads, page_size, D/2]")
    pages, kv_heads, page_size, half = kc.shape
    _sizes(page_size, kv_heads, 2 * half)
    u8, index = torch.uint8, kc.get_device()
    shapes = _shapes(pages, page_size, kv_heads, 2 * half)
    if not (_is(kc, shapes[0], u8, index) and _is(ks, shapes[1], u8, index) and
            _is(vc, shapes[2], u8, index) and _is(vs, shapes[3], u8, index)):
        for t, name, shape in zip(cache, KVCache._fields, shapes):
            _need(t, name, shape, u8, kc.device)
    return _Cache(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, page_size,
                  kv_heads, 2 * half, _held(k_exp, 32), _held(v_exp, 32)), index


def _vectors(t, name, shape, dtype, index):
    """A [tokens, heads, D] tensor with unit stride along D and free others."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along its last dim")


def _plain(t, name, shape, dtype, index):
    if not _is(t, shape, dtype, index):
        _need(t, name, shape, dtype, torch.device("cuda", index))


def append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_exp: int = 0,
           v_exp: int = 0, mode: int = MODE_ADAPTIVE) -> KVCache:
    """Quantize k and v ([tokens, kv_heads, D], fp32 or bf16, unit stride along
    D, other strides multiples of 16 bytes: slices of a fused projection are
    fine) into the cache's slots (int64 [tokens], all different; a slot outside
    the cache is skipped).  Returns the cache, which is written in place."""
    st = _kv_call.append(cache, k, v, slots, k_exp, v_exp, mode)
    if st == 0:
        return cache
    if st:
        _check("if4_kv_append", st)
    c, index = _cache(cache, k_exp, v_exp)
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a 3-D tensor [tokens, kv_heads, D]")
    shape = (k.shape[0], c.kv_heads, c.head_dim)
    _vectors(k, "k", shape, k.dtype, index)
    _vectors(v, "v", shape, k.dtype, index)
    _plain(slots, "slots", shape[:1], torch.int64, index)
    (kt, kh, _), (vt, vh, _) = k.stride(), v.stride()
    st = lib.if4_kv_append(c, k.data_ptr(), v.data_ptr(), _dtype_code(k.dtype), shape[0], kt, kh,
                           vt, vh, slots.data_ptr(), _held(mode, 32), _raw_stream(index))
    if st:
        _check("if4_kv_append", st)
    return cache


def read(cache: KVCache, slots: torch.Tensor, k_exp: int = 0, v_exp: int = 0,
         dtype=torch.bfloat16, out=None):
    """Values of the cache's slots (int64 [tokens]): (k, v), each [tokens,
    kv_heads, D] of `dtype` (bf16 or fp32).  A slot outside the cache reads as
    zeros.  `out` may pass preallocated (k, v)."""
    if out is None and (dtype is torch.bfloat16 or dtype is torch.float32):
        kv = _kv_call.read(cache, slots, k_exp, v_exp, dtype is torch.bfloat16)
        if type(kv) is tuple:
            return kv
        if kv:
            _check("if4_kv_read", kv)
    c, index = _cache(cache, k_exp, v_exp)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D tensor")
    _plain(slots, "slots", slots.shape, torch.int64, index)
    shape = (slots.shape[0], c.kv_heads, c.head_dim)
    if out is None:
        k = torch.empty(shape, dtype=dtype, device=slots.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        if not isinstance(k, torch.Tensor):
            raise ValueError("out must be two tensors (k, v)")
        _plain(k, "k", shape, k.dtype, index)
        _plain(v, "v", shape, k.dtype, index)
    st = lib.if4_kv_read(c, slots.data_ptr(), shape[0], k.data_ptr(), v.data_ptr(),
                         _dtype_code(k.dtype), _raw_stream(index))
    if st:
        _check("if4_kv_read", st)
    return k, v


def attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
              q_starts: torch.Tensor, *, max_q: int, max_len=None, scale=None, k_exp: int = 0,
              v_exp: int = 0, causal: bool = True, window: int = 0, sinks: int = 0, out=None,
              workspace=None) -> torch.Tensor:
    """Attention of the newest tokens of a batch of sequences over the cache.

    q [total_q, heads, D] bf16 (unit stride along D) holds the sequences'
    newest tokens one after another, sequence b in rows q_starts[b] ..
    q_starts[b + 1] - 1 (int32 [batch + 1]); seq_lens (int32 [batch]) counts
    the tokens that each has in the cache, these included; page_table (int32
    [batch, pages of the longest]) names their pages.  max_q: the most rows of
    any sequence.  max_len: about how long the longest is (default: what the
    page table has room for); it only steers how the work is split.

    Rows past a sequence's first max_q and rows of no sequence (a padded batch)
    are not written: they keep what `out` holds, and are unset without one.

    A row at position p sees key j iff j <= p (causal) and, with a window, j >
    p - window or j < sinks.  Rows that see no key give zeros.  scale defaults
    to 1/sqrt(D).  Returns [total_q, heads, D] bf16; `out` may pass it
    preallocated, `workspace` a uint8 tensor of workspace_bytes()."""
    if out is None and workspace is None:
        r = _kv_call.attention(q, cache, page_table, seq_lens, q_starts, max_q, max_len, scale, k_exp,
                               v_exp, causal, window, sinks)
        if type(r) is int:
            _check("if4_kv_attention", r)
        elif r is not None:
            return r
    c, index = _cache(cache, k_exp, v_exp)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a 3-D tensor [total_q, heads, D]")
    shape = total, heads, dim = q.shape
    _vectors(q, "q", (total, heads, c.head_dim), torch.bfloat16, index)
    if heads == 0 or heads % c.kv_heads:
        raise ValueError(f"heads ({heads}) must be a multiple of kv_heads ({c.kv_heads})")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a 2-D tensor [batch, pages]")
    batch, width = page_table.shape
    _plain(page_table, "page_table", (batch, width), torch.int32, index)
    _plain(seq_lens, "seq_lens", (batch,), torch.int32, index)
    _plain(q_starts, "q_starts", (batch + 1,), torch.int32, index)
    scale = dim ** -0.5 if scale is None else float(scale)
    if not 0 <= scale < math.inf:
        raise ValueError("scale must be finite and not negative")
    if window < 0 or sinks < 0 or (not causal and (window or sinks)):
        raise ValueError("window and sinks must not be negative, and need causal")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    else:
        _vectors(out, "out", shape, torch.bfloat16, index)
    (qt, qh, _), (ot, oh, _) = q.stride(), out.stride()
    a = _Attention(q.data_ptr(), out.data_ptr(), qt, qh, ot, oh, page_table.data_ptr(), width,
                   seq_lens.data_ptr(), q_starts.data_ptr(), batch, total, heads, _held(max_q, 64),
                   width * c.page_size if max_len is None else _held(max_len, 64),
                   _held(window, 64), _held(sinks, 64), scale, 1 if causal else 0)
    need = lib.if4_kv_attention_workspace(c, a)
    if need < 0:
        _check("if4_kv_attention", -need)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or \
                workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
                workspace.numel() < need:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {q.device}")
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = lib.if4_kv_attention(c, a, workspace.data_ptr() if need else None, need,
                              _raw_stream(index))
    if st:
        _check("if4_kv_attention", st)
    return out


def workspace_bytes(cache: KVCache, *, total_q: int, heads: int, batch: int, max_q: int,
                    max_len: int, window: int = 0, sinks: int = 0) -> int:
    """Bytes that are enough for every attention() of such a cache with no more of
    these sizes, whatever its window: a program that captures calls in a graph, or
    makes many, allocates them once."""
    c, _ = _cache(cache, 0, 0)
    sizes = dict(batch=batch, total_q=total_q, heads=heads, max_q=max_q, max_len=max_len,
                 window=window, sinks=sinks)
    a = _Attention(scale=1.0, causal=1, **{name: _held(n, 64) for name, n in sizes.items()})
    need = lib.if4_kv_attention_workspace_most(c, a)
    if need < 0:
        _check("if4_kv_attention_workspace_most", -need)
    return need
