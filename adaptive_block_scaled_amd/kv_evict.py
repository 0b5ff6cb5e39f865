"""Eviction from the paged IF4 KV cache by accumulated attention weight: the Python binding
of include/if4_kv_evict.h.

`accumulate` adds the attention weights of a call's newest tokens to a running sum for
every cached token and kv head ("mass", fp32 [sequences, kv_heads, width]); it takes
what kv_cache.attention takes.  `select` names the tokens to keep: the first ones, the
latest ones, and those with the largest sums.  `compact` copies their K and V into other
pages; the old ones are free afterwards, and the sequence goes on with the new pages and
min(its length, keep) tokens.  Every kv head keeps tokens of its own.

As in the rest of the binding, arguments are checked and marshalled here, all work
runs in the HIP kernels of libif4.so on torch's current stream, and nothing records a
gradient.
"""
import ctypes
import math

import torch

from .if4 import _check, _on, lib
from .kv_cache import KVCache, _Attention, _Cache, _cache, _held, _kv_call, _plain, _raw_stream, _vectors

EXPORTS = ("if4_kv_weights", "if4_kv_weights_workspace", "if4_kv_weights_workspace_most", "if4_kv_select",
           "if4_kv_select_workspace", "if4_kv_compact")


class _Mass(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("in_stride_row", ctypes.c_int64), ("in_stride_head", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_stride_row", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
                ("rows", ctypes.c_void_p), ("mass_rows", ctypes.c_int64), ("width", ctypes.c_int64)]


def _declare():
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    cache, args, mass = (ctypes.POINTER(t) for t in (_Cache, _Attention, _Mass))
    lib.if4_kv_weights.restype = ci
    lib.if4_kv_weights.argtypes = [cache, args, mass, vp, i64, vp]
    for f in (lib.if4_kv_weights_workspace, lib.if4_kv_weights_workspace_most):
        f.restype = i64
        f.argtypes = [cache, args]
    lib.if4_kv_select.restype = ci
    lib.if4_kv_select.argtypes = [mass, vp, i64, i64, i64, i64, i64, vp, vp, i64, vp]
    lib.if4_kv_select_workspace.restype = i64
    lib.if4_kv_select_workspace.argtypes = [mass, i64, i64, i64]
    lib.if4_kv_compact.restype = ci
    lib.if4_kv_compact.argtypes = [cache, vp, i64, vp, i64, i64, vp, i64, vp]


_declare()
_kv_call.bind_evict(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
    "if4_kv_weights", "if4_kv_weights_workspace", "if4_kv_select", "if4_kv_select_workspace", "if4_kv_compact")))


def _sums(t, name, kv_heads, device, rows=None, width=None):
    """A [sequences, kv_heads, width] fp32 tensor with unit stride along its last dim."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dim() != 3 or t.shape[1] != kv_heads or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must have shape ({'sequences' if rows is None else rows}, {kv_heads}, width), "
                         f"not {tuple(t.shape)}")
    if width is not None and t.shape[2] < width:
        raise ValueError(f"{name} must be {width} wide at least, not {t.shape[2]}")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be torch.float32, not {t.dtype}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along its last dim")


def _apart(t):
    """Whether rows along the last dim do not overlap: strides as of some order of the first two."""
    (n, h, w), (sn, sh, _) = t.shape, t.stride()
    return (n <= 1 or sn >= w) and (h <= 1 or sh >= w) and \
        (n <= 1 or h <= 1 or sn >= sh * (h - 1) + w or sh >= sn * (n - 1) + w)


def _mass(mass, out, rows, batch, device):
    if rows is not None:
        _plain(rows, "rows", (batch,), torch.int32, device.index)
    elif mass.shape[0] < batch:
        raise ValueError(f"mass must have a row for each of {batch} sequences, or rows be given")
    if out is not None and not _apart(out):
        raise ValueError("the sums' rows must not overlap")
    return _Mass(mass.data_ptr(), mass.stride(0), mass.stride(1), None if out is None else out.data_ptr(),
                 0 if out is None else out.stride(0), 0 if out is None else out.stride(1),
                 None if rows is None else rows.data_ptr(), mass.shape[0], mass.shape[2])


def accumulate(mass: torch.Tensor, q: torch.Tensor, cache: KVCache, page_table: torch.Tensor,
               seq_lens: torch.Tensor, q_starts: torch.Tensor, *, max_q: int, max_len=None, rows=None,
               scale=None, k_exp: int = 0, causal: bool = True, window: int = 0, sinks: int = 0, out=None,
               workspace=None) -> torch.Tensor:
    """Add the attention weights of the newest tokens to the sums of the tokens that they
    attend to, per kv head.  q .. sinks are those of kv_cache.attention.

    mass (fp32 [sequences, kv_heads, width], unit stride along its last dim) has sequence
    b's sums in row rows[b] (int32 [batch], all different; default: row b; a row outside
    leaves the sequence out).  The tokens whose rows of q these are start from nothing, older
    ones from what mass holds.  Tokens at and past `width` have no sum.  Returns `out`, by
    default mass itself, written in place; a new `out` of mass's shape gets the sums of the
    call's sequences and keeps the rest.  `workspace` may pass a uint8 tensor of
    workspace_bytes()."""
    if workspace is None:
        to = mass if out is None else out
        st = _kv_call.weights(mass, to, rows, q, cache, page_table, seq_lens, q_starts, max_q, max_len, scale, k_exp,
                              causal, window, sinks)
        if st == 0:
            return to
        if st:
            _check("if4_kv_weights", st)
    c, index = _cache(cache, k_exp, 0)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a 3-D tensor [total_q, heads, D]")
    total, heads, dim = q.shape
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
    _sums(mass, "mass", c.kv_heads, q.device)
    if out is None:
        out = mass
    elif out is not mass:
        _sums(out, "out", c.kv_heads, q.device, mass.shape[0], mass.shape[2])
    m = _mass(mass, out, rows, batch, q.device)
    qt, qh, _ = q.stride()
    a = _Attention(q.data_ptr(), None, qt, qh, 0, 0, page_table.data_ptr(), width, seq_lens.data_ptr(),
                   q_starts.data_ptr(), batch, total, heads, _held(max_q, 64),
                   width * c.page_size if max_len is None else _held(max_len, 64),
                   _held(window, 64), _held(sinks, 64), scale, 1 if causal else 0)
    need = lib.if4_kv_weights_workspace(c, a)
    if need < 0:
        _check("if4_kv_weights", -need)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or \
                workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {q.device}")
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = _on(index, lib.if4_kv_weights, c, a, m, workspace.data_ptr() if need else None, need, _raw_stream(index))
    if st:
        _check("if4_kv_weights", st)
    return out


def workspace_bytes(cache: KVCache, *, total_q: int, heads: int, batch: int, max_q: int, max_len: int) -> int:
    """Bytes that are enough for every accumulate() of such a cache with no more of these
    sizes: a program that captures calls in a graph, or makes many, allocates them once."""
    c, _ = _cache(cache, 0, 0)
    sizes = dict(batch=batch, total_q=total_q, heads=heads, max_q=max_q, max_len=max_len)
    a = _Attention(scale=1.0, causal=1, **{name: _held(n, 64) for name, n in sizes.items()})
    need = lib.if4_kv_weights_workspace_most(c, a)
    if need < 0:
        _check("if4_kv_weights_workspace_most", -need)
    return need


def select(mass: torch.Tensor, seq_lens: torch.Tensor, keep: int, *, recent: int = 0, sinks: int = 0, rows=None,
           out=None, mass_out=None, workspace=None) -> torch.Tensor:
    """Positions of the `keep` tokens of each sequence and kv head to keep, int32 [batch,
    kv_heads, keep], ascending: the first `sinks`, the last `recent`, and the ones with the
    largest sums between them (equal ones: the earlier); all of a sequence that has no more,
    then -1.  Row rows[b] of mass belongs to sequence b, as in accumulate; seq_lens counts
    its tokens.  `mass_out` (mass itself is fine) gets the kept tokens' sums in
    places 0, 1, ..; `out` may pass the positions preallocated, `workspace` a uint8 tensor of
    select_workspace_bytes()."""
    if out is None and workspace is None:
        kept = _kv_call.select(mass, seq_lens, keep, recent, sinks, rows, mass_out)
        if type(kept) is int:
            _check("if4_kv_select", kept)
        elif kept is not None:
            return kept
    if not isinstance(mass, torch.Tensor) or mass.dim() != 3 or not mass.is_cuda:
        raise ValueError("mass must be a CUDA tensor [sequences, kv_heads, width]")
    kv_heads, dev = mass.shape[1], mass.device
    _sums(mass, "mass", kv_heads, dev)
    if kv_heads == 0:
        raise ValueError("mass must have kv heads")
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be a 1-D tensor [batch]")
    batch = seq_lens.shape[0]
    _plain(seq_lens, "seq_lens", (batch,), torch.int32, dev.index)
    keep, recent, sinks = int(keep), int(recent), int(sinks)
    if keep < 0 or recent < 0 or sinks < 0 or recent + sinks > keep:
        raise ValueError("keep, recent and sinks must not be negative, nor recent + sinks more than keep")
    if mass_out is not None and mass_out is not mass:
        _sums(mass_out, "mass_out", kv_heads, dev, mass.shape[0], min(keep, mass.shape[2]))
    if out is None:
        out = torch.empty((batch, kv_heads, keep), dtype=torch.int32, device=dev)
    else:
        _plain(out, "out", (batch, kv_heads, keep), torch.int32, dev.index)
    m = _mass(mass, mass_out, rows, batch, dev)
    need = lib.if4_kv_select_workspace(m, batch, kv_heads, keep)
    if need < 0:
        _check("if4_kv_select", -need)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != dev or workspace.dtype != torch.uint8 or \
                not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {dev}")
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = _on(dev.index, lib.if4_kv_select, m, seq_lens.data_ptr(), batch, kv_heads, keep, recent, sinks, out.data_ptr(),
             workspace.data_ptr() if need else None, need, _raw_stream(dev.index))
    if st:
        _check("if4_kv_select", st)
    return out


def select_workspace_bytes(mass: torch.Tensor, batch: int, keep: int) -> int:
    """Bytes of workspace that select() takes for such sums (0 unless they are long)."""
    m = _Mass(mass_rows=mass.shape[0], width=mass.shape[2])
    need = lib.if4_kv_select_workspace(m, batch, mass.shape[1], keep)
    if need < 0:
        _check("if4_kv_select_workspace", -need)
    return need


def compact(cache: KVCache, page_table: torch.Tensor, kept: torch.Tensor, new_table: torch.Tensor) -> KVCache:
    """Copy K and V of the kept tokens (select's result) from the pages of page_table (int32
    [batch, pages]) to places 0, 1, .. of new_table's (int32 [batch, pages]), which must
    be other ones.  Returns the cache, which is written in place."""
    st = _kv_call.compact(cache, page_table, kept, new_table, 0)
    if st == 0:
        return cache
    if st:
        _check("if4_kv_compact", st)
    c, index = _cache(cache, 0, 0)
    for t, name, dims in ((page_table, "page_table", 2), (kept, "kept", 3), (new_table, "new_table", 2)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must be a {dims}-D tensor")
    batch, width = page_table.shape
    _plain(page_table, "page_table", (batch, width), torch.int32, index)
    _plain(kept, "kept", (batch, c.kv_heads, kept.shape[2]), torch.int32, index)
    _plain(new_table, "new_table", (batch, new_table.shape[1]), torch.int32, index)
    st = _on(index, lib.if4_kv_compact, c, page_table.data_ptr(), width, kept.data_ptr(), batch, kept.shape[2],
             new_table.data_ptr(), new_table.shape[1], _raw_stream(index))
    if st:
        _check("if4_kv_compact", st)
    return cache
