"""Plain 64-bit reference of the paged IF4 KV cache, on the CPU: the cache's
layouts, the values of its bytes, and attention over them, written from the
definitions in include/if4_kv.h with tables and loops."""
import math

import numpy as np

E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)])
E4M3[127] = np.nan
FP4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
INT4 = np.array([i * 6 / 7 for i in range(8)] + [-i * 6 / 7 for i in range(8)])


def row_values(codes, scales, exp):
    """64-bit values of IF4 rows: codes [..., D/2], scales [..., D/16]."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    sc = np.repeat(scales, 16, -1)
    base = np.where(sc >= 128, INT4[nib], FP4[nib])
    return base * E4M3[sc & 127] * 2.0 ** exp


def v_rows(v_codes, v_scales):
    """V of a cache as rows [pages, heads, page_size, ...]."""
    p, h, tiles, _, _, nb = v_codes.shape
    codes = v_codes.transpose(0, 1, 2, 4, 3, 5).reshape(p, h, tiles * 16, 16 * nb)
    scales = v_scales.transpose(0, 1, 2, 4, 3).reshape(p, h, tiles * 16, -1)
    return np.ascontiguousarray(codes), np.ascontiguousarray(scales)


def slot_rows(cache, part, slot):
    """(codes [heads, D/2], scales [heads, D/16]) of one slot, found byte by byte."""
    page_size = cache["k_codes"].shape[2]
    p, o = slot // page_size, slot % page_size
    if part == "k":
        return cache["k_codes"][p, :, o], cache["k_scales"][p, :, o]
    codes = cache["v_codes"][p, :, o // 16, :, o % 16]  # [heads, 16, D/32]
    return codes.reshape(codes.shape[0], -1), cache["v_scales"][p, :, o // 16, :, o % 16]


def attention(q, cache, table, lens, starts, scale, k_exp, v_exp, causal=True, window=0, sinks=0):
    """(out, bound) in 64 bits, [rows, heads, D]: what the operator defines and
    how far a right kernel may be from it, from its stated arithmetic:

      * K and V operands: an INT4 value is fl16(|q| fl16(6 s'/7)), within
        2 * 2^-11 relative, and no finer than 2^-15 2^E (the smallest fp16
        number is 2^-24, operands carry 2^-9); FP4 values are exact;
      * q: exact down to 2^-24 of the row's largest magnitude;
      * scores: fp32 sums of D products (fewer than D + 8 roundings of 2^-24),
        exp2's argument rounded once more, exp2 within 2 units of 2^-23;
      * probabilities: fp16 (2^-11 relative, 2^-25 absolute against a largest
        one of at least 1), sums in fp32 (a rounding of 2^-24 for each key);
      * the output: one rounding to bf16 (2^-9 relative).
    """
    rows, heads, dim = q.shape
    kv_heads, page_size = cache["k_codes"].shape[1:3]
    group = heads // kv_heads
    vc, vs = v_rows(cache["v_codes"], cache["v_scales"])
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        n = int(min(max(n, 0), table.shape[1] * page_size))
        first, t_b = starts[b], starts[b + 1] - starts[b]
        if n == 0:
            continue
        j = np.arange(n)
        pages, offs = table[b, j // page_size], j % page_size
        for h in range(kv_heads):
            k = row_values(cache["k_codes"][pages, h, offs], cache["k_scales"][pages, h, offs], k_exp)
            v = row_values(vc[pages, h, offs], vs[pages, h, offs], v_exp)
            for i in range(t_b):
                pos = n - t_b + i
                seen = np.full(n, True)
                if causal:
                    seen &= j <= pos
                if window:
                    seen &= (j > pos - window) | (j < sinks)
                if not seen.any():
                    continue
                ks, vv = k[seen], v[seen]
                for m in range(h * group, (h + 1) * group):
                    x = q[first + i, m]
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = (ks @ x) * scale
                        e = np.exp(s - s.max())
                        p = e / e.sum()
                        y = p @ vv
                        grain_k, grain_v = 2.0 ** (k_exp - 15), 2.0 ** (v_exp - 15)
                        absx = np.abs(x)
                        ds = scale * (np.abs(ks) @ absx * (2.0 ** -10 + (dim + 8) * 2.0 ** -24)
                                      + grain_k * absx.sum()
                                      + 2.0 ** -24 * absx.max() * np.abs(ks).sum(1))
                        dp = np.expm1(ds.max() + np.abs(s).max() * 2.0 ** -22 + 2.0 ** -21)
                        rel = 2 * dp + 2.0 ** -11 + 2.0 ** -10 + 2 * seen.sum() * 2.0 ** -24
                        far = (p @ np.abs(vv)) * rel + grain_v + \
                            seen.sum() * 2.0 ** -25 * np.abs(vv).max(0)
                    out[first + i, m] = y
                    bound[first + i, m] = np.abs(y) * 2.0 ** -9 + far * (1 + 2.0 ** -8) + 1e-38
    return out, bound
