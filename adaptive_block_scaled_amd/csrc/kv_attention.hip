// Attention over the paged IF4 KV cache for gfx950 (definition and layouts in
// include/if4_kv.h).
//
// Rows.  The rows of a tile are (token, query head of one kv head's group)
// pairs, r = token * group + head in group, so that every decoded key serves
// the whole group: a decode step with a group of 8 fills 8 rows, a chunk of
// prompt fills tiles of tokens x heads.
//
// One pass.  S^T = K Q^T puts a query row in a matrix-core column: a lane
// holds scores of one row only, its running maximum m and partial sum l stay
// in registers, and the probabilities come out of the accumulators in the
// operand order of O^T = V^T P^T (the order of the keys inside one
// product is free as long as V's operand uses the same).  m is raised only
// where a score exceeds it by more than 8 (in powers of two): p <= 2^8 is far
// inside fp16, and most units then need neither a cross-lane maximum nor a
// rescale of the accumulators.
//
// Small probabilities.  fp16 holds what is 2^-14 in full and what is 2^-25 at all.  With
// few rows m lies 7 below the largest score, and small ones keep 7 bits more.  The
// other kernels leave it out: there one wave adds up to all keys of a row to one
// accumulator, in which the matrix core rounds what is below 2^-24 of it, and with
// probabilities finer than that the products and l no longer round alike (2^20 keys
// of one value, the first with 2^24.5 times the others' weight: 0.5% low).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "if4_internal.h"
#include "kv_internal.h"
#include "kv_operand.h"

namespace if4 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// (lambdas that hold a kernel's state have to be inlined, whatever their size)
#define KV_INLINE __attribute__((always_inline))

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kUnit = 32;             // keys that a wave takes at once
constexpr float kLowest = -3.0e38f;   // running maximum before any key
constexpr float kSlack = 8.0f;        // how far scores may exceed the largest one it was raised to
constexpr float kLift = 7.0f;         // how far it lies below that one, few rows
constexpr int kMaxLen = 0x3FFFFF00;   // keys of a sequence
constexpr int kHidden = 0x3FFFFF80;   // first key of a step that no row sees

struct Args {
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_st, q_sh, o_st, o_sh;
    const int32_t *page_table, *seq_lens, *q_starts;
    int64_t table_stride;
    float *part_o, *part_ml;  // splits > 1: [splits][rows_all][D], [..][2]
    int64_t rows_all;         // rows of q times heads, or see part_row
    int total_q, max_q, pages, kv_heads, heads, batch_heads, row_tiles, splits, split_units;
    int batch, compact;  // see item_of
    int join_tokens;     // see part_row
    int above, upto;  // sequences with rows of a head in (above, upto] are this launch's
    int causal, window, sinks;
    Divisor tiles;  // of 16 tokens in a page
    Divisor group;  // query heads of a kv head
    float q_scale;  // scale * log2(e)
    int k_exp;      // E of K plus the 9 of its operands
    float v_mul;    // 2^(E of V + 9)
};

// One sequence, as a workgroup sees it.
struct Sequence {
    int first_row, rows;  // rows of q
    int len, pos0;        // keys, position of its first row
    const int32_t* table;
    // tile rows of a kv head, those of the first max_q rows of q
    __device__ __forceinline__ int tile_rows(const Args& p) const {
        return (rows < p.max_q ? rows : p.max_q) * (int)p.group.n;
    }
};

__device__ __forceinline__ Sequence sequence_of(const Args& p, int b) {
    Sequence s;
    int q0 = p.q_starts[b], q1 = p.q_starts[b + 1];
    q0 = q0 < 0 ? 0 : q0 > p.total_q ? p.total_q : q0;
    q1 = q1 < q0 ? q0 : q1 > p.total_q ? p.total_q : q1;
    s.first_row = q0;
    s.rows = q1 - q0;
    int64_t room = p.table_stride * p.tiles.n * 16;
    room = room < kMaxLen ? room : kMaxLen;
    const int64_t len = p.seq_lens[b];
    s.len = (int)(len < 0 ? 0 : len > room ? room : len);
    s.pos0 = s.len - s.rows;
    s.table = p.page_table + b * p.table_stride;
    return s;
}

// The units of keys that rows at positions lo .. hi see: the first `sink`
// units, then those from `start` on.
struct KeyUnits {
    int sink, start, n;
    __device__ __forceinline__ int operator()(int i) const {
        return i < sink ? i : i - sink + start;
    }
};

__device__ __forceinline__ KeyUnits key_units(const Args& p, int len, int lo, int hi, int unit) {
    const int end = p.causal ? (hi + 1 < len ? hi + 1 : len) : len;
    KeyUnits u = {0, 0, 0};
    if (end <= 0) return u;
    int start = 0;
    if (p.window) {
        start = lo - p.window + 1;
        start = start < 0 ? 0 : start;
    }
    u.start = start / unit;
    const int s = p.sinks < start ? p.sinks : start;
    u.sink = (s + unit - 1) / unit;
    u.sink = u.sink < u.start ? u.sink : u.start;
    u.n = u.sink + (end + unit - 1) / unit - u.start;
    return u;
}

// Units that a split takes.  By the length hint, the same for every sequence,
// so that workgroups take equally long and a short sequence has fewer of
// them, unless this one is too long for that.
__device__ __forceinline__ int units_per_split(const Args& p, int n) {
    const int own = (n + p.splits - 1) / p.splits;
    return own > p.split_units ? own : p.split_units;
}

// A sum that no split has: the join leaves the row of out as it is.
constexpr float kLeftAlone = -1.0f;

// First row of a sequence in the partial sums: that of q, and in the launch of
// sequences with few rows (see launches_of) one of join_tokens rows for each of the batch.
__device__ __forceinline__ int part_row(const Args& p, const Sequence& s, int b) {
    return p.join_tokens == 0 ? s.first_row : b * p.join_tokens;
}

// Tile rows row0 .. last_row of a split that nothing is computed for, of the sequence whose
// partial sums start at row `first`.  Without keys (sum 0) the join skips the split.
__device__ __forceinline__ void mark(const Args& p, int first, int head, int row0, int last_row,
                                     int split, float sum) {
    for (int r = row0 + threadIdx.x; r <= last_row; r += blockDim.x) {
        const int t = (int)p.group.into(r), g = r - t * (int)p.group.n;
        const int64_t at = split * p.rows_all + (int64_t)(first + t) * p.heads +
                           head * (int)p.group.n + g;
        *reinterpret_cast<f32x2*>(p.part_ml + 2 * at) = f32x2{kLowest, sum};
    }
}
__device__ __forceinline__ void mark_empty(const Args& p, int first, int head, int row0,
                                           int last_row, int split) {
    mark(p, first, head, row0, last_row, split, 0.0f);
}

// Rows of q that no workgroup computes, for a join that goes over all rows: those
// before the first sequence and behind the last one, and those past max_q of each.
__device__ __forceinline__ void mark_ends(const Args& p, int head, int first, int end) {
    mark(p, 0, head, 0, first * (int)p.group.n - 1, 0, kLeftAlone);
    mark(p, end, head, 0, (p.total_q - end) * (int)p.group.n - 1, 0, kLeftAlone);
}
__device__ __forceinline__ int last_token(const Args& p) {
    const Sequence s = sequence_of(p, p.batch - 1);
    return s.first_row + s.rows;
}
// (by the first workgroup of a sequence and head; item_of has marked the ends of a
// compact grid, in which a sequence without rows has no workgroup)
__device__ __forceinline__ void mark_unowned(const Args& p, const Sequence& s, int b, int head) {
    mark(p, s.first_row, head, s.tile_rows(p), s.rows * (int)p.group.n - 1, 0, kLeftAlone);
    if (p.compact || (b > 0 && b < p.batch - 1)) return;
    mark_ends(p, head, b == 0 ? s.first_row : 0,
              b == p.batch - 1 ? s.first_row + s.rows : p.total_q);
}

// What a workgroup of the tiles of many rows does: a row tile of a (sequence, head)
// pair, a split of its keys.  Pairs are fastest and the last row tiles, which see
// the most keys, come first.  Where chunks differ in length (compact) the tiles that
// hold rows and their splits that hold keys are counted, 64 sequences at a time, and
// come first and without gaps: a grid of max_q for every sequence would be empty for
// the most part, and workgroups that leave at once hold up those behind them, of which
// each place on the chip gets its share in turn (6 chunks of 100 to 700 tokens over
// 1000 to 6000 keys, 32 heads, D = 128: 279 us, so 202; 24 of 1 to 61, 61 to 5003 keys, 21
// heads, D = 256: 106, so 91).  Sequences of another launch have none; their rows are marked for
// the join here.
struct Item {
    int b, head, row_tile, split;
    int splits;  // of this sequence that may hold keys; the others are marked by split 0
};
template <int kRows, bool kTurn>
__device__ __forceinline__ bool item_of(const Args& p, Item& it) {
    const int index = blockIdx.x;
    it.splits = p.splits;
    if (!p.compact) {
        const int rest = index / p.batch_heads;
        // (workgroups 8 apart share an XCD: turned by 3 per row tile and split, those
        // of one long sequence are spread over all of them)
        const int bh = (index + (kTurn ? 3 * rest : 0)) % p.batch_heads;
        it.row_tile = p.row_tiles - 1 - rest % p.row_tiles;
        it.split = rest / p.row_tiles;
        it.b = bh / p.kv_heads;
        it.head = bh - it.b * p.kv_heads;
        return true;
    }
    const int lane = threadIdx.x & 63;
    int splits = 0;  // of this lane's sequence
    const auto count = [&](int i) KV_INLINE {
        if (i >= p.batch) return 0;
        const Sequence s = sequence_of(p, i);
        const int rows = s.rows * (int)p.group.n, n = (s.tile_rows(p) + kRows - 1) / kRows;
        // (not less than any row tile has, see units_per_split)
        splits = ((s.len + 63) / 64 + p.split_units - 1) / p.split_units;
        splits = splits < p.splits ? splits > 0 ? splits : 1 : p.splits;
        return rows > p.above && rows <= p.upto ? (n < p.row_tiles ? n : p.row_tiles) * splits : 0;
    };
    const auto up_to = [&](int n) KV_INLINE {  // inclusive sums over the lanes
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int other = __shfl_up(n, d);
            n += lane >= d ? other : 0;
        }
        return n;
    };
    it.head = index % p.kv_heads;
    if (p.splits > 1 && index < p.kv_heads)
        mark_ends(p, it.head, sequence_of(p, 0).first_row, last_token(p));
    if (p.above > 0 && p.splits > 1 && index < p.kv_heads)
        for (int i = threadIdx.x; i < p.batch; i += blockDim.x) {
            const Sequence s = sequence_of(p, i);
            if (s.rows * (int)p.group.n > p.above) continue;
            for (int t = 0; t < s.rows; t++)
                for (int g = 0; g < (int)p.group.n; g++) {
                    const int64_t at = (int64_t)(s.first_row + t) * p.heads +
                                       it.head * (int)p.group.n + g;
                    *reinterpret_cast<f32x2*>(p.part_ml + 2 * at) = f32x2{kLowest, kLeftAlone};
                }
        }
    // the sums of all before sequences from .. from + 63, the last ones first
    const int last = (p.batch - 1) & ~63;
    int total = 0;
    for (int i = 0; i < last; i += 64)
        total += __builtin_amdgcn_readlane(up_to(count(i + lane)), 63);
    int from = last, sums = up_to(count(from + lane)) + total;
    int t = __builtin_amdgcn_readlane(sums, 63) - 1 - index / p.kv_heads;
    if (t < 0) return false;
    while (t < total) {
        from -= 64;
        if (from < 0) return false;
        sums = up_to(count(from + lane));
        total -= __builtin_amdgcn_readlane(sums, 63);
        sums += total;
    }
    const int before = __builtin_popcountll(__builtin_amdgcn_ballot_w64(sums <= t));
    if (before > 63) return false;
    t -= before ? __builtin_amdgcn_readlane(sums, before - 1) : total;
    it.b = from + before;
    if (it.b >= p.batch) return false;
    it.splits = __builtin_amdgcn_readlane(splits, before);
    // row tiles fastest
    const int all = __builtin_amdgcn_readlane(sums, before) -
                    (before ? __builtin_amdgcn_readlane(sums, before - 1) : total);
    const int tiles = all / it.splits;
    // (where q_starts do not ascend, chunks can overlap and the sums pass 31 bits: no
    // item outside the batch or its tiles comes of that)
    if (t < 0 || t >= all || tiles <= 0) return false;
    it.split = t / tiles;
    it.row_tile = t - it.split * tiles;
    return it.split < it.splits && it.row_tile < p.row_tiles;
}

// First keys of the steps of `step` keys that every row of a tile sees whole:
// at most `hi`, and at least `lo` or at most `sink`.
struct WholeSteps {
    int lo, hi, sink;
    __device__ __forceinline__ WholeSteps(const Args& p, int len, int pos_lo, int pos_hi,
                                          int step) {
        const int n = p.causal && pos_lo + 1 < len ? pos_lo + 1 : len;
        hi = n - step;
        lo = p.window ? pos_hi - p.window + 1 : -1;
        sink = p.sinks - step;
    }
    __device__ __forceinline__ bool operator()(int key0) const {
        return (key0 <= hi) & ((key0 >= lo) | (key0 <= sink));
    }
};

// Cache tile (16 tokens) of one kv head that holds keys 16 n .. 16 n + 15 of
// a sequence; n past its last key gives some valid tile.  Made in two steps,
// so that the page table's entry can be on its way long before its use.
struct TileRef {
    int page;
    uint32_t rest;  // tile in the page
};
// (page: its place in the sequence's row of the table)
__device__ __forceinline__ TileRef tile_ref_of(const Args& p, const Sequence& s, int n) {
    const int last = s.len > 0 ? (s.len - 1) >> 4 : 0;
    const uint32_t m = (uint32_t)(n < last ? n : last);
    const uint32_t i = p.tiles.into(m);
    return {(int)i, m - i * p.tiles.n};
}
__device__ __forceinline__ TileRef tile_ref(const Args& p, const Sequence& s, int n) {
    const TileRef r = tile_ref_of(p, s, n);
    // (constant address space: a scalar load, whatever stores are around)
    typedef const __attribute__((address_space(4))) int32_t* Table;
    return {((Table)(uintptr_t)s.table)[r.page], r.rest};
}
// (all tiles of a cache, pages x kv heads x tiles of a page, fit 31 bits)
__device__ __forceinline__ uint32_t cache_tile(const Args& p, int head, TileRef r) {
    const int last = p.pages - 1;
    int page = r.page < last ? r.page : last;
    page = page > 0 ? page : 0;
    return (uint32_t)(page * p.kv_heads + head) * p.tiles.n + r.rest;
}

// 4, as a value that the compiler cannot fold (see HighBytes).
__device__ __forceinline__ uint32_t opaque_four(const Args& p) {
    return 4u + ((uint32_t)p.total_q >> 31);
}

// f(0), f(1) .. f(n - 1) with constants.
template <int n, int i = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
    if constexpr (i < n) {
        f(std::integral_constant<int, i>{});
        each<n, i + 1>(f);
    }
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const f32x2 t = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(t, half2v));
}

// sum + both fp16 values of h (v_dot2 adds two exactly): l sums what O's products see.
__device__ __forceinline__ float add_half2(uint32_t h, float sum) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2v, h),
                                  __builtin_bit_cast(half2v, 0x3C003C00u), sum, false);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 t = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(t, bf16x2));
}

// What a row's scores are multiplied by: q was divided by 2^e.  Kept finite
// and above zero, so that a hidden key's score of -inf stays -inf.
__device__ __forceinline__ float score_factor(const Args& p, int e) {
    const float c = __builtin_ldexpf(p.q_scale, p.k_exp + e);
    return __builtin_fminf(__builtin_fmaxf(c, 1.17549435e-38f), 3.40282347e38f);
}

// How far a score x (of a row with this factor) lies above m: the exponent of its
// probability, so that what does not exceed the slack is inside fp16 at any size of m.
__device__ __forceinline__ float above(float x, float factor, float m) {
    return __builtin_fmaf(x, factor, -m);
}

// Token, row of q and query head of tile row r (the last row's past the end).
struct RowPlace {
    int token;
    int64_t row, head;
    __device__ __forceinline__ RowPlace(const Args& p, const Sequence& s, int kv_head, int r,
                                        int rows) {
        const int rc = r < rows ? r : rows - 1;
        token = (int)p.group.into(rc);
        row = s.first_row + token;
        head = kv_head * (int)p.group.n + (rc - token * (int)p.group.n);
    }
};

// Scores of keys that a row does not see become -inf.  x[i] is the score of key
// first + 8 (i / 4) + i % 4 for the row at position pos.
__device__ __forceinline__ void hide(const Args& p, int len, int pos, int first,
                                     f32x16& x) {
    const int last = p.causal && pos < len - 1 ? pos : len - 1;
    const int hi = last - first;
#pragma unroll
    for (int i = 0; i < 16; i++)
        x[i] = 8 * (i >> 2) + (i & 3) <= hi ? x[i] : -__builtin_inff();
    if (p.window) {
        const int lo = pos - p.window - first, sink = p.sinks - first;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int c = 8 * (i >> 2) + (i & 3);
            x[i] = ((c > lo) | (c < sink)) ? x[i] : -__builtin_inff();
        }
    }
}

// q in fp16, divided by the power of two that brings a row's largest magnitude
// into [1, 2): exact down to 2^-24 of it.  A row with an infinity or NaN becomes
// NaN as a whole, and so do its scores, whatever the keys.  The largest
// magnitude is found on the bits of the bf16 values, two at a time.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
struct RowMagnitude {
    u16x2 top = {0, 0};
    __device__ __forceinline__ void take(const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; j++)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[j] & 0x7FFF7FFFu));
    }
    // largest bits of this lane
    __device__ __forceinline__ int bits() const { return top[0] > top[1] ? top[0] : top[1]; }
};
// of a row whose largest magnitude has these bits
struct RowScale {
    int e;
    float by;
    __device__ __forceinline__ RowScale(int bits) {
        e = bits == 0 ? 0 : (bits >> 7) - 127;
        by = bits < 0x7F80 ? __builtin_ldexpf(1.0f, -e) : __uint_as_float(0x7FC00000u);
    }
    __device__ __forceinline__ half8 operand(const uint4& v) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            h[j] = pack_half(__uint_as_float(w[j] << 16) * by,
                             __uint_as_float(w[j] & 0xFFFF0000u) * by);
        return __builtin_bit_cast(half8, make_uint4(h[0], h[1], h[2], h[3]));
    }
};
__device__ __forceinline__ int larger(int a, int b) { return a > b ? a : b; }

// ---------------------------------------------------------------------------
// Few rows (a decode step, short chunks): tiles of 16 * kBlocks rows.
//
// Each wave takes its own units of 32 keys, with its own m, l and O, and reads
// their codes straight from memory into operands: v_mfma_f32_16x16x32_f16 of
// K lane l = (key l % 16, quarter l / 16 of D) is a contiguous 1 KB of the
// cache per load at D = 128, and so is V's, lane l = (piece l % 16, tokens
// 4 (l / 16) ..).  Nothing is shared but the scale tables, until the four
// waves' results are joined in LDS.
//
// Bound by memory while the rows are few: 64 sequences of 3001 to 12289 keys, 64
// heads, D = 128 (566 MB): 119 us = 4.8 TB/s of a copy's 5.2; 4 of 100003 to 131071
// (533 MB): 111 us = 4.8 TB/s.  One sequence of 4097 keys is latency: 7 us for a
// launch, the lengths, the page table, the codes, one after another.  With 32 rows per
// tile two waves of a SIMD hide less of it: 16 chunks of 4 tokens over 8192 keys, 64
// heads: 56 us, 2.8 TB/s.
template <int D>
struct UnitCodes {
    uint32_t k[2][D / 32], v[2][D / 32];
    uint32_t ks[2], vs[2];

    template <typename T>
    __device__ static __forceinline__ void words(const uint8_t* src, T& dst) {
        if constexpr (D == 64) {
            const uint2 a = *reinterpret_cast<const uint2*>(src);
            dst[0] = a.x;
            dst[1] = a.y;
        } else {
#pragma unroll
            for (int i = 0; i < D / 128; i++) {
                const uint4 a = *reinterpret_cast<const uint4*>(src + 16 * i);
                dst[4 * i] = a.x;
                dst[4 * i + 1] = a.y;
                dst[4 * i + 2] = a.z;
                dst[4 * i + 3] = a.w;
            }
        }
    }
    __device__ __forceinline__ void load_k(const Args& p, const uint32_t (&at)[2], int lane) {
        const uint32_t code = (lane & 15) * (D / 2) + (lane >> 4) * (D / 8);
        const uint32_t scale = (lane & 15) * (D / 16) + (lane >> 4) * (D / 64);
#pragma unroll
        for (int t = 0; t < 2; t++) {
            words(p.k_codes + (uint64_t)at[t] * (8 * D) + code, k[t]);
            const uint8_t* src = p.k_scales + (uint64_t)at[t] * D + scale;
            if constexpr (D == 64)
                ks[t] = *src;
            else if constexpr (D == 128)
                ks[t] = *reinterpret_cast<const uint16_t*>(src);
            else
                ks[t] = *reinterpret_cast<const uint32_t*>(src);
        }
    }
    __device__ __forceinline__ void load_v(const Args& p, const uint32_t (&at)[2], int lane) {
        const uint32_t code = (lane & 15) * (D / 2) + (lane >> 4) * (D / 8);
        const uint32_t scale = (lane & 15) * D / 256 * 16 + (lane >> 4) * 4;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            words(p.v_codes + (uint64_t)at[t] * (8 * D) + code, v[t]);
            vs[t] = *reinterpret_cast<const uint32_t*>(p.v_scales + (uint64_t)at[t] * D + scale);
        }
    }
};

template <int D, int kBlocks>
struct FewRows {
    // Waves per SIMD that the registers are held to: single-token calls are
    // bound by the latency of their loads (64 sequences of 3-12k keys: 154 us
    // with two, 145 with three, 144 with four; 16 rows at D = 128 use 128
    // registers).
    static constexpr int kOccupancy = D * kBlocks <= 128 ? 4 : 2;
    static constexpr int kRows = 16 * kBlocks;
    static constexpr int kPad = D + 4;
    static constexpr int kLds = kScaleTableBytes + kWaves * 16 * kPad * 4 + 2 * kWaves * kRows * 4;
};

template <int D, int kBlocks>
__global__ void __launch_bounds__(kThreads, (FewRows<D, kBlocks>::kOccupancy))
few_rows_kernel(const Args p) {
    constexpr int kRows = 16 * kBlocks, kPad = D + 4, M = D / 16;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint2* const tables = reinterpret_cast<uint2*>(smem);
    float* const joined = reinterpret_cast<float*>(smem + kScaleTableBytes);
    float* const joined_m = joined + kWaves * 16 * kPad;
    float* const joined_l = joined_m + kWaves * kRows;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // (sequence, kv head) fastest: workgroups are dealt to the 8 XCDs in turn,
    // so the row tiles and splits of one pair share an XCD's L2 wherever the
    // number of pairs is a multiple of 8
    const int bh = blockIdx.x % p.batch_heads, rest = blockIdx.x / p.batch_heads;
    const int row_tile = rest % p.row_tiles, split = rest / p.row_tiles;
    const int b = bh / p.kv_heads, head = bh - b * p.kv_heads;

    const Sequence s = sequence_of(p, b);
    const int row0 = row_tile * kRows, rows = s.tile_rows(p);
    if (p.splits > 1 && p.join_tokens == 0 && split == 0 && row_tile == 0)
        mark_unowned(p, s, b, head);
    if (row0 >= rows || s.rows * (int)p.group.n > p.upto) return;
    const uint32_t four = opaque_four(p);
    const int last_row = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
    const int pos_lo = s.pos0 + (int)p.group.into(row0), pos_hi = s.pos0 + (int)p.group.into(last_row);
    const KeyUnits units = key_units(p, s.len, pos_lo, pos_hi, kUnit);
    const int per = units_per_split(p, units.n);
    const int begin = split * per;
    const int end = begin + per < units.n ? begin + per : units.n;
    if (p.splits > 1 && begin >= end) {
        mark_empty(p, part_row(p, s, b), head, row0, last_row, split);
        return;
    }
    fill_scale_tables(tables, tid, kThreads);

    // this lane's row of each block, its q as operands, and what it sees:
    // keys <= see_hi that are > see_lo or < sinks
    half8 q[kBlocks][D / 32];
    float factor[kBlocks];
    int see_hi[kBlocks], see_lo[kBlocks];
#pragma unroll
    for (int nr = 0; nr < kBlocks; nr++) {
        const int r = row0 + 16 * nr + (lane & 15);
        const int rc = r < rows ? r : rows - 1;
        const int t = (int)p.group.into(rc), g = rc - t * (int)p.group.n;
        const uint16_t* src = p.q + (s.first_row + t) * p.q_st +
                              (int64_t)(head * (int)p.group.n + g) * p.q_sh + (lane >> 4) * (D / 4);
        uint4 raw[D / 32];
        RowMagnitude a;
#pragma unroll
        for (int i = 0; i < D / 32; i++) {
            raw[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
            a.take(raw[i]);
        }
        int bits = a.bits();
        bits = larger(bits, __shfl_xor(bits, 16));
        const RowScale scale(larger(bits, __shfl_xor(bits, 32)));
#pragma unroll
        for (int i = 0; i < D / 32; i++) q[nr][i] = scale.operand(raw[i]);
        factor[nr] = score_factor(p, scale.e);
        const int pos = s.pos0 + t;
        see_hi[nr] = p.causal && pos < s.len - 1 ? pos : s.len - 1;
        see_lo[nr] = p.window ? pos - p.window : -1;
    }

    f32x4 o[M][kBlocks];
    float m[kBlocks], l[kBlocks];
#pragma unroll
    for (int nr = 0; nr < kBlocks; nr++) {
        m[nr] = kLowest;
        l[nr] = 0.0f;
#pragma unroll
        for (int d = 0; d < M; d++) o[d][nr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();

    UnitCodes<D> c;
    // one unit; `next`: the cache tiles whose codes are asked for as soon as
    // this unit's are decoded
    auto compute = [&](int unit, const uint32_t (&next)[2]) {
        const int key0 = unit * kUnit;
        f32x4 acc[2][kBlocks];
#pragma unroll
        for (int t = 0; t < 2; t++) {
#pragma unroll
            for (int nr = 0; nr < kBlocks; nr++) acc[t][nr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < D / 32; i += 2) {
                KGroup group;
                group.unpack(c.k[t][i], c.k[t][i + 1],
                             k_scale(tables, (c.ks[t] >> (4 * i)) & 0xFFu), four);
                const half8 a[2] = {group.operand<0>(), group.operand<1>()};
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int nr = 0; nr < kBlocks; nr++)
                        acc[t][nr] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            a[j], q[nr][i + j], acc[t][nr], 0, 0, 0);
            }
        }
        c.load_k(p, next, lane);
        // does every row of the tile see every key of the unit?
        const bool all = key0 + kUnit <= s.len && (!p.causal || key0 + kUnit - 1 <= pos_lo) &&
                         (!p.window || key0 > pos_hi - p.window || key0 + kUnit <= p.sinks);
        const int lane_key = key0 + 4 * (lane >> 4);
        uint4 prob[kBlocks];
#pragma unroll
        for (int nr = 0; nr < kBlocks; nr++) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = acc[j >> 2][nr][j & 3];
            if (!all) {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int key = lane_key + 16 * (j >> 2) + (j & 3);
                    const bool seen = key <= see_hi[nr] && (key > see_lo[nr] || key < p.sinks);
                    x[j] = seen ? x[j] : -__builtin_inff();
                }
            }
            float top = x[0];
#pragma unroll
            for (int j = 1; j < 8; j++) top = __builtin_fmaxf(top, x[j]);
            if (__builtin_amdgcn_ballot_w64(above(top, factor[nr], m[nr]) > kSlack + kLift) != 0) {
                top = __builtin_fmaxf(above(top, factor[nr], kLift), m[nr]);
                top = __builtin_fmaxf(top, __shfl_xor(top, 16));
                top = __builtin_fmaxf(top, __shfl_xor(top, 32));
                const float alpha = __builtin_amdgcn_exp2f(m[nr] - top);
                m[nr] = top;
                l[nr] *= alpha;
#pragma unroll
                for (int d = 0; d < M; d++)
#pragma unroll
                    for (int i = 0; i < 4; i++) o[d][nr][i] *= alpha;
            }
#pragma unroll
            for (int j = 0; j < 8; j++)
                x[j] = __builtin_amdgcn_exp2f(above(x[j], factor[nr], m[nr]));
            // (a unit's sum first: added pair by pair, small ones to a large l lose more)
            uint32_t h[4];
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                h[j] = pack_half(x[2 * j], x[2 * j + 1]);
                sum = add_half2(h[j], sum);
            }
            l[nr] += sum;
            prob[nr] = make_uint4(h[0], h[1], h[2], h[3]);
        }
        VPiece<D> v[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            GroupScale sc[4];
            VPiece<D>::look_up(tables, c.vs[t], sc);
            v[t].unpack(c.v[t], sc, four);
        }
        const uint32_t vs[2] = {c.vs[0], c.vs[1]};
        c.load_v(p, next, lane);
        each<M>([&](auto dim) {
            constexpr int d = decltype(dim)::value;
            const half8 a = __builtin_bit_cast(
                half8, make_uint4(v[0].template pair<d, 0>(), v[0].template pair<d, 1>(),
                                  v[1].template pair<d, 0>(), v[1].template pair<d, 1>()));
#pragma unroll
            for (int nr = 0; nr < kBlocks; nr++)
                o[d][nr] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    a, __builtin_bit_cast(half8, prob[nr]), o[d][nr], 0, 0, 0);
        });
        // NaN values of V (decoded as zeros): into the rows that see them
        if (__builtin_amdgcn_ballot_w64((nan_bytes(vs[0]) | nan_bytes(vs[1])) != 0) != 0) {
#pragma unroll 1
            for (int j = 0; j < 8; j++) {
                const uint32_t byte = ((j >> 2 ? vs[1] : vs[0]) >> (8 * (j & 3))) & 0x7Fu;
                const uint64_t bad = __builtin_amdgcn_ballot_w64(byte == 0x7Fu);
#pragma unroll 1
                for (int quarter = 0; quarter < 4; quarter++) {
                    const uint32_t pieces = (uint32_t)(bad >> (16 * quarter)) & 0xFFFFu;
                    const int key = key0 + 16 * (j >> 2) + 4 * quarter + (j & 3);
#pragma unroll
                    for (int nr = 0; nr < kBlocks; nr++) {
                        const bool seen =
                            key <= see_hi[nr] && (key > see_lo[nr] || key < p.sinks);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const bool hit = seen && (pieces >> (4 * (lane >> 4) + i) & 1u);
#pragma unroll
                            for (int d = 0; d < M; d++)
                                o[d][nr][i] = hit ? __uint_as_float(0x7FC00000u) : o[d][nr][i];
                        }
                    }
                }
            }
        }
    };

    int i = begin + wave;
    if (i < end) {
        const auto refs = [&](int j, TileRef (&r)[2]) {
            const int u = units(j < end ? j : end - 1);
            r[0] = tile_ref(p, s, 2 * u);
            r[1] = tile_ref(p, s, 2 * u + 1);
        };
        const auto tiles = [&](const TileRef (&r)[2], uint32_t (&at)[2]) {
            at[0] = cache_tile(p, head, r[0]);
            at[1] = cache_tile(p, head, r[1]);
        };
        TileRef r[2];
        uint32_t at[2];
        refs(i, r);
        tiles(r, at);
        c.load_k(p, at, lane);
        c.load_v(p, at, lane);
        refs(i + kWaves, r);
#pragma unroll 1
        for (; i < end; i += kWaves) {
            tiles(r, at);
            refs(i + 2 * kWaves, r);
            compute(units(i), at);
        }
    }

    // join the waves
#pragma unroll
    for (int nr = 0; nr < kBlocks; nr++) {
        l[nr] += __shfl_xor(l[nr], 16);
        l[nr] += __shfl_xor(l[nr], 32);
        if (lane < 16) {
            joined_m[wave * kRows + 16 * nr + lane] = m[nr];
            joined_l[wave * kRows + 16 * nr + lane] = l[nr];
        }
    }
#pragma unroll
    for (int nr = 0; nr < kBlocks; nr++) {
        if (nr) __syncthreads();
#pragma unroll
        for (int i2 = 0; i2 < 4; i2++) {
            float* dst = joined + (wave * 16 + (lane & 15)) * kPad + (4 * (lane >> 4) + i2) * M;
#pragma unroll
            for (int d = 0; d < M; d += 4)
                *reinterpret_cast<f32x4*>(dst + d) = f32x4{o[d][nr][i2], o[d + 1][nr][i2],
                                                           o[d + 2][nr][i2], o[d + 3][nr][i2]};
        }
        __syncthreads();
        // thread: row tid / 16 of the block, dims (tid % 16) * M ..
        const int rr = tid >> 4, r = row0 + 16 * nr + rr;
        if (r < rows) {
            float mw[kWaves], top = kLowest, sum = 0.0f, acc[M];
#pragma unroll
            for (int w = 0; w < kWaves; w++) {
                mw[w] = joined_m[w * kRows + 16 * nr + rr];
                top = __builtin_fmaxf(top, mw[w]);
            }
#pragma unroll
            for (int d = 0; d < M; d++) acc[d] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; w++) {
                const float f = __builtin_amdgcn_exp2f(mw[w] - top);
                sum = __builtin_fmaf(f, joined_l[w * kRows + 16 * nr + rr], sum);
                const float* src = joined + (w * 16 + rr) * kPad + (tid & 15) * M;
#pragma unroll
                for (int d = 0; d < M; d++) acc[d] = __builtin_fmaf(f, src[d], acc[d]);
            }
            const int t = (int)p.group.into(r), g = r - t * (int)p.group.n;
            const int64_t row = s.first_row + t, hd = head * (int)p.group.n + g;
            if (p.splits == 1) {
                const float f = sum == 0.0f ? 0.0f : p.v_mul / sum;
                uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * p.o_st + hd * p.o_sh +
                                                            (tid & 15) * M);
#pragma unroll
                for (int d = 0; d < M; d += 2) dst[d / 2] = pack_bf16(acc[d] * f, acc[d + 1] * f);
            } else {
                const int64_t at = split * p.rows_all + (part_row(p, s, b) + t) * (int64_t)p.heads + hd;
                float* dst = p.part_o + at * D + (tid & 15) * M;
#pragma unroll
                for (int d = 0; d < M; d++) dst[d] = acc[d];
                if ((tid & 15) == 0) {
                    p.part_ml[2 * at] = top;
                    p.part_ml[2 * at + 1] = sum;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// What the two kernels with 32 rows per wave share: a lane holds one row (row =
// lane % 32 of its wave), half = lane / 32.

// q of a row as the operands of D / 16 products: words 2t + half of 8 dims.
template <int D, typename Word>
__device__ __forceinline__ void make_q(const Args& p, Word&& word, half8 (&q)[D / 16],
                                       float& factor) {
    uint4 w[D / 16];
    RowMagnitude a;
#pragma unroll
    for (int i = 0; i < D / 16; i++) {
        w[i] = word(i);
        a.take(w[i]);
    }
    const RowScale scale(larger(a.bits(), __shfl_xor(a.bits(), 32)));
#pragma unroll
    for (int i = 0; i < D / 16; i++) q[i] = scale.operand(w[i]);
    factor = score_factor(p, scale.e);
}
template <int D>
__device__ __forceinline__ void take_q(const Args& p, const Sequence& s, int head, int r, int rows,
                                       int half, half8 (&q)[D / 16], float& factor, int& pos) {
    const RowPlace at(p, s, head, r, rows);
    const uint16_t* src = p.q + at.row * p.q_st + at.head * p.q_sh + half * 8;
    make_q<D>(p, [&](int i) { return *reinterpret_cast<const uint4*>(src + 16 * i); }, q, factor);
    pos = s.pos0 + at.token;
}

// q of a tile of kRows rows, on its way through LDS.  Each row is asked for by
// neighbouring lanes, 16 bytes each, and taken from LDS by the lanes that need it as
// operands: straight from memory the 32 rows of a wave's operand would be 32 lines
// of 32 bytes (D = 256: 13200 cycles until q and the first codes are there, so 7800;
// 2 prompts of 4096 tokens at D = 128 583 -> 580 us.  Many rows, whose workgroups ask
// for half as much and have no cycles to spare for LDS, are 3% faster without).
// In LDS (kRows * 2 D bytes of a tile buffer) a row's 16-byte words are permuted so that
// a column of words lies in different banks.
template <int D, int kRows, int kThreadsOf>
struct TileQ {
    static constexpr int kWords = D / 8, kPasses = kRows * kWords / kThreadsOf;
    typedef u32x4 Words[kPasses];
    __device__ static __forceinline__ uint32_t place(int r, int word) {
        const int turn = (D == 64 ? r >> 1 : r) & (kWords < 16 ? kWords - 1 : 15);
        return (uint32_t)(r * kWords + (word ^ turn)) * 16;
    }
    __device__ static __forceinline__ void ask(const Args& p, const Sequence& s, int head,
                                               int row0, int rows, int tid, Words& raw) {
#pragma unroll
        for (int i = 0; i < kPasses; i++) {
            const RowPlace at(p, s, head, row0 + (i * kThreadsOf + tid) / kWords, rows);
            raw[i] = *reinterpret_cast<const u32x4*>(p.q + at.row * p.q_st + at.head * p.q_sh +
                                                     tid % kWords * 8);
        }
    }
    __device__ static __forceinline__ void put(uint8_t* lds, int tid, const Words& raw) {
#pragma unroll
        for (int i = 0; i < kPasses; i++)
            *reinterpret_cast<u32x4*>(
                lds + place((i * kThreadsOf + tid) / kWords, tid % kWords)) = raw[i];
    }
    // row r of the tile
    __device__ static __forceinline__ void take(const Args& p, const uint8_t* lds, int r, int half,
                                                half8 (&q)[D / 16], float& factor) {
        make_q<D>(
            p, [&](int i) { return *reinterpret_cast<const uint4*>(lds + place(r, 2 * i + half)); },
            q, factor);
    }
};
// Position of tile row r (the last row's past the end).
__device__ __forceinline__ int position_of(const Args& p, const Sequence& s, int r, int rows) {
    return s.pos0 + (int)p.group.into(r < rows ? r : rows - 1);
}

__device__ __forceinline__ bool sees(const Args& p, int len, int pos, int key) {
    return (key <= pos || !p.causal) & (key < len) &
           (!p.window || key > pos - p.window || key < p.sinks);
}

// Probabilities of 32 keys, 16 of them in this lane, as the operands of O's
// products.  l sums what those see, the fp16 values (v_dot2 adds two exactly).
__device__ __forceinline__ void probabilities(const f32x16& x, float factor, float m, float& l,
                                              uint4 (&prob)[2]) {
    float e[16];
#pragma unroll
    for (int i = 0; i < 16; i++)
        e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], factor, -m));
    uint32_t h[8];
    float sum[2] = {l, 0.0f};  // two short chains
#pragma unroll
    for (int i = 0; i < 8; i++) {
        h[i] = pack_half(e[2 * i], e[2 * i + 1]);
        sum[i & 1] = add_half2(h[i], sum[i & 1]);
    }
    l = sum[0] + sum[1];
    prob[0] = make_uint4(h[0], h[1], h[2], h[3]);
    prob[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

// A row's result: B blocks of 32 dims, accumulator i of block d in V-piece row
// 8 (i / 4) + 4 half + i % 4 (mod 16), so that a lane holds 2 B dims of 8 pieces.
template <int D, int B>
__device__ __forceinline__ void store_row(const Args& p, const Sequence& s, int head, int r,
                                          int rows, int half, int split, int part_of_o,
                                          f32x16 (&o)[B], float m, float l, uint32_t poisoned) {
    l += __shfl_xor(l, 32);
    if (r >= rows) return;
    const RowPlace at(p, s, head, r, rows);
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int piece = (8 * (i >> 2) + 4 * half + (i & 3)) & 15;
        const bool hit = poisoned >> (piece * D / 256) & 1;
#pragma unroll
        for (int d = 0; d < B; d++) o[d][i] = hit ? __uint_as_float(0x7FC00000u) : o[d][i];
    }
    const int first = part_of_o * 2 * B;
    if (p.splits == 1) {
        const float f = l == 0.0f ? 0.0f : p.v_mul / l;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int piece = 8 * (i >> 2) + 4 * half + (i & 3);
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at.row * p.o_st + at.head * p.o_sh +
                                                        piece * (D / 16) + first);
#pragma unroll
            for (int d = 0; d < B; d++) dst[d] = pack_bf16(o[d][i] * f, o[d][i + 8] * f);
        }
    } else {
        const int64_t to = split * p.rows_all + at.row * p.heads + at.head;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int piece = 8 * (i >> 2) + 4 * half + (i & 3);
            f32x2* dst = reinterpret_cast<f32x2*>(p.part_o + to * D + piece * (D / 16) + first);
#pragma unroll
            for (int d = 0; d < B; d++) dst[d] = f32x2{o[d][i], o[d][i + 8]};
        }
        if (half == 0 && part_of_o == 0)
            *reinterpret_cast<f32x2*>(p.part_ml + 2 * to) = f32x2{m, l};
    }
}

// ---------------------------------------------------------------------------
// Many rows (33 to 128, D <= 128): tiles of 128 rows, 4 waves of 32 rows each.
//
// The four waves share K and V: each decodes one 16-token cache tile of every
// 64 keys into double-buffered LDS tiles in the order of the operands of
// v_mfma_f32_32x32x16_f16, so that every operand is one contiguous 1 KB
// ds_read_b128 and every ds_write covers whole banks.
//
// Operand order.  K, block of 32 keys, step t: lane (key, half h) holds word
// 2t + h (8 dims) of its key.  V, 16 keys, block b of 32 rows: row r is dim
// M (r % 16) + 2b + r / 16 with M = D/16 (the pieces of the cache's V are rows
// apart), lane (row, h) holds keys 4h .. 4h + 3 and 8 + 4h .. 11 + 4h: the
// order in which S^T's accumulators hold the probabilities.
//
// Steps of 32 keys are pipelined: while the matrix cores compute the scores of
// step k + 1, the VALU turns those of step k into probabilities, and while
// they add step k to O, it decodes the next tile.  4 chunks of 16 tokens over 16384
// keys, 64 heads, D = 128 (128 rows each): 72 us with the join, 478 TFLOP/s, 1.1
// TB/s.  No pipe is full: the matrix cores are busy 30% of the time and the VALU 44%, and
// of a wave's time 36% go into waiting to issue and 26% into barriers, LDS and loads.
template <int D>
struct ManyRows {
    static constexpr int kTile = 64 * D * 2;  // bytes of K or V of 64 keys
    static constexpr int kFlags = kScaleTableBytes + 4 * kTile;
    static constexpr int kLds = kFlags + 2 * kWaves * 4;
};

// Workgroup barrier that orders LDS only: global loads in flight (the codes
// of the next tiles) are not waited for.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 4 : 2) many_rows_kernel(const Args p) {
    constexpr int kRows = 128, T = D / 16, B = D / 32, M = D / 16;
    constexpr int kTile = ManyRows<D>::kTile;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint2* const tables = reinterpret_cast<uint2*>(smem);
    uint8_t* const k_lds = smem + kScaleTableBytes;
    uint8_t* const v_lds = k_lds + 2 * kTile;
    uint32_t* const flags = reinterpret_cast<uint32_t*>(smem + ManyRows<D>::kFlags);

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Item it;
    if (!item_of<kRows, false>(p, it)) return;
    const int b = __builtin_amdgcn_readfirstlane(it.b);
    const int head = __builtin_amdgcn_readfirstlane(it.head);
    const int row_tile = __builtin_amdgcn_readfirstlane(it.row_tile);
    const int split = __builtin_amdgcn_readfirstlane(it.split);
    const int own_splits = __builtin_amdgcn_readfirstlane(it.splits);

    const Sequence s = sequence_of(p, b);
    const int row0 = row_tile * kRows, rows = s.tile_rows(p);
    if (p.splits > 1 && split == 0 && row_tile == 0) mark_unowned(p, s, b, head);
    if (row0 >= rows) return;
    const uint32_t four = opaque_four(p);
    const int last_row = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
    const int pos_lo = s.pos0 + (int)p.group.into(row0), pos_hi = s.pos0 + (int)p.group.into(last_row);
    const KeyUnits units = key_units(p, s.len, pos_lo, pos_hi, 64);
    const int per = units_per_split(p, units.n);
    const int begin = split * per;
    const int end = begin + per < units.n ? begin + per : units.n;
    if (split == 0)
        for (int i = own_splits; i < p.splits; i++) mark_empty(p, s.first_row, head, row0, last_row, i);
    if (p.splits > 1 && begin >= end) {
        mark_empty(p, s.first_row, head, row0, last_row, split);
        return;
    }
    fill_scale_tables(tables, tid, kThreads);

    half8 q[T];
    float factor, m = kLowest, l = 0.0f;
    int pos;
    take_q<D>(p, s, head, row0 + 32 * wave + (lane & 31), rows, half, q, factor, pos);
    uint32_t poisoned = 0;  // groups of O that are NaN
    f32x16 o[B], x[2];
#pragma unroll
    for (int d = 0; d < B; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0.0f;

    // this lane's codes of its wave's cache tile: K (key lane % 16, quarter
    // lane / 16 of D), V (piece lane % 16, tokens 4 quarter ..); V's quarters
    // are dealt so that each half wave writes whole 16-byte pieces
    const int kq = lane >> 4, vq = (kq & 1) * 2 + (kq >> 1);
    const uint32_t k_at = (lane & 15) * (D / 2) + kq * (D / 8);
    const uint32_t v_at = (lane & 15) * (D / 2) + vq * (D / 8);
    const uint32_t ks_at = (lane & 15) * (D / 16) + kq * (D / 64);
    const uint32_t vs_at = (lane & 15) * D / 256 * 16 + vq * 4;
    uint8_t* const k_to = k_lds + ((wave >> 1) * T + kq * (D / 64)) * 1024 +
                          (16 * (wave & 1) + (lane & 15)) * 16;
    uint8_t* const v_to =
        v_lds + wave * B * 1024 + ((vq & 1) * 32 + (lane & 15)) * 16 + (vq >> 1) * 8;

    uint32_t kw[D / 32], vw[D / 32], ks, vs;
    auto ref = [&](int i) { return tile_ref(p, s, 4 * units(i < end ? i : end - 1) + wave); };
    auto load_k = [&](uint64_t at) {
        UnitCodes<D>::words(p.k_codes + at * (8 * D) + k_at, kw);
        const uint8_t* src = p.k_scales + at * D + ks_at;
        if constexpr (D == 64)
            ks = *src;
        else
            ks = *reinterpret_cast<const uint16_t*>(src);
    };
    auto load_v = [&](uint64_t at) {
        UnitCodes<D>::words(p.v_codes + at * (8 * D) + v_at, vw);
        vs = *reinterpret_cast<const uint32_t*>(p.v_scales + at * D + vs_at);
    };
    auto decode_k = [&](int buf) {
#pragma unroll
        for (int w = 0; w < D / 32; w += 2) {
            KGroup group;
            group.unpack(kw[w], kw[w + 1], k_scale(tables, (ks >> (4 * w)) & 0xFFu), four);
            const half8 a[2] = {group.operand<0>(), group.operand<1>()};
#pragma unroll
            for (int j = 0; j < 2; j++)
                *reinterpret_cast<half8*>(k_to + buf * kTile + (w >> 1) * 1024 + j * 512) = a[j];
        }
    };
    auto decode_v = [&](int buf) {
        VPiece<D> v;
        GroupScale sc[4];
        VPiece<D>::look_up(tables, vs, sc);
        v.unpack(vw, sc, four);
        each<M>([&](auto dim) {
            constexpr int d = decltype(dim)::value;
            *reinterpret_cast<uint2*>(v_to + buf * kTile + (d >> 1) * 1024 + (d & 1) * 256) =
                make_uint2(v.template pair<d, 0>(), v.template pair<d, 1>());
        });
        const uint64_t bad = __builtin_amdgcn_ballot_w64(nan_bytes(vs) != 0);
        if (lane == 0) flags[buf * kWaves + wave] = bad != 0;
    };
    // scores of 32 keys
    auto scores = [&](f32x16& to, int buf, int kb) {
        const uint8_t* src = k_lds + buf * kTile + kb * T * 1024 + lane * 16;
#pragma unroll
        for (int i = 0; i < 16; i++) to[i] = 0.0f;
#pragma unroll
        for (int t = 0; t < T; t++)
            to = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                *reinterpret_cast<const half8*>(src + t * 1024), q[t], to, 0, 0, 0);
    };
    // hides what a row does not see, and raises m where it has to
    const WholeSteps whole(p, s.len, pos_lo, pos_hi, 32);
    auto settle = [&](f32x16& sc, int key0) {
        if (!whole(key0)) hide(p, s.len, pos, key0 + 4 * half, sc);
        float top = sc[0];
#pragma unroll
        for (int i = 1; i < 16; i++) top = __builtin_fmaxf(top, sc[i]);
        top *= factor;
        if (__builtin_amdgcn_ballot_w64(top > m + kSlack) == 0) return;
        top = __builtin_fmaxf(top, m);
        top = __builtin_fmaxf(top, __shfl_xor(top, 32));
        const float alpha = __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < B; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) o[d][i] *= alpha;
    };
    uint4 prob[2];
    auto accumulate = [&](int buf, int kb) {
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int d = 0; d < B; d++) {
                const half8 a = *reinterpret_cast<const half8*>(
                    v_lds + buf * kTile + ((2 * kb + i) * B + d) * 1024 + lane * 16);
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                    a, __builtin_bit_cast(half8, prob[i]), o[d], 0, 0, 0);
            }
    };
    // NaN values of V (decoded as zeros) of a 64-key tile: the groups that turn
    // NaN in the rows that see them
    auto poison = [&](int u) {
#pragma unroll 1
        for (int j = 0; j < 4 * T; j++) {  // 16-token tile j / T, group j % T
            const uint64_t at = cache_tile(p, head, tile_ref(p, s, 4 * u + j / T));
            const uint8_t* src = p.v_scales + at * D + (j % T) * 16;
#pragma unroll 1
            for (int t = 0; t < 16; t++) {
                const int key = 64 * u + 16 * (j / T) + t;
                const bool hit = (src[t] & 0x7F) == 0x7F && sees(p, s.len, pos, key);
                poisoned |= (uint32_t)hit << (j % T);
            }
        }
    };

    __syncthreads();
    if (begin < end) {
        uint32_t at = cache_tile(p, head, ref(begin));
        load_k(at);
        load_v(at);
        decode_k(0);
        at = cache_tile(p, head, ref(begin + 1));
        load_k(at);
        decode_v(0);
        load_v(at);
        TileRef next = ref(begin + 2);
        lds_barrier();
        scores(x[0], 0, 0);
        settle(x[0], 64 * units(begin));
#pragma unroll 1
        for (int i = begin; i < end; i++) {
            const int buf = (i - begin) & 1, u = units(i);
            at = cache_tile(p, head, next);
            next = ref(i + 3);
            // keys 0 .. 31 of the tile
            scores(x[1], buf, 1);
            probabilities(x[0], factor, m, l, prob);
            accumulate(buf, 0);
            decode_k(buf ^ 1);
            load_k(at);
            settle(x[1], 64 * u + 32);
            lds_barrier();
            // keys 32 .. 63
            const uint4 f = *reinterpret_cast<const uint4*>(flags + buf * kWaves);
            scores(x[0], buf ^ 1, 0);
            probabilities(x[1], factor, m, l, prob);
            accumulate(buf, 1);
            decode_v(buf ^ 1);
            load_v(at);
            if (__builtin_amdgcn_readfirstlane((f.x | f.y) | (f.z | f.w)) != 0) poison(u);
            if (i + 1 < end) settle(x[0], 64 * units(i + 1));
            lds_barrier();
        }
    }

    store_row<D, B>(p, s, head, row0 + 32 * wave + (lane & 31), rows, half, split, 0, o, m, l,
                    poisoned);
}

// ---------------------------------------------------------------------------
// Prompts (more than 128 rows): tiles of 256 rows, 8 waves of 32.
//
// Two waves share a SIMD, wave w and w + 4, and take turns: while one issues
// the products of a step (A: scores of step k + 1, O of step k, 512 cycles of
// matrix core at D = 128), the other does the VALU work of its step (B:
// probabilities of step k + 1), with a barrier between the phases; waves 4-7 run
// one phase behind.  Each wave decodes a quarter of a K or V tile in one of its
// A phases, between the products.  With c = 64-key tile, phases of waves 0-3:
// A(2c) = 4c, B(2c) = 4c + 1, ..; of waves 4-7 one later.
//   * waves 0-3 decode V of tile c + 1 in A(2c), phase 4c.  V of tile c - 1, in
//     the same buffer, was last read in A(2c - 1) of waves 4-7, phase 4c - 1; V of
//     tile c + 1 is first read in A(2c + 2), phase 4c + 4.
//   * waves 4-7 decode K of tile c + 2 in A(2c + 1), phase 4c + 3.  K of tile c,
//     in the same buffer, was last read (as step 2c + 1) in A(2c) of waves 4-7,
//     phase 4c + 1; K of tile c + 2 is first read in A(2c + 2), phase 4c + 4.
// Operands and their order are those of many_rows_kernel.  The decode's work is cut
// into even slices of about four instructions behind each product: with a group's
// unpacking in one piece, D = 128 was 1% slower, D = 256 3%.
//
// 2048 new of 16384 tokens, 64 heads, D = 128: 975 us, 1057 TFLOP/s (with all waves
// in step, as in many_rows_kernel, 1161 us); D = 64: 611 us, 844 TFLOP/s, at a
// power-limited clock of about 2 GHz.  No pipe is full: the matrix cores are busy 53% of the
// time, and the VALU issues in 57%, with the products and 6.5 other instructions for each
// (decode 2, softmax 3); of a wave's time 44% are issue, 36% waiting to issue and 20%
// waiting at barriers and for LDS.  The phases are not alike, a tile's decode lies in
// two of four, and each ends for all waves with its longest.  A workgroup's start (lengths,
// pages, codes and q one after another, then code that no cache holds yet) takes about
// 5 us.
constexpr int kPairWaves = 8, kPairThreads = 64 * kPairWaves;

template <int D>
struct PromptTile {
    static constexpr int kTile = 64 * D * 2;  // bytes of K or V of 64 keys
    static constexpr int kFlags = kScaleTableBytes + 4 * kTile;
    static constexpr int kLds = kFlags + 2 * kWaves * 4;
};

// Both halves of a workgroup run this, each in code of its own from beginning to
// end (kLate: waves 4-7): with shared ends around two loops the register
// allocator spilled 21 registers at D = 128; apart they need 210 of 256.
template <int D, bool kLate>
__device__ __forceinline__ void prompt_rows(const Args& p) {
    typedef PromptTile<D> Tile;
    // products of a step: T for the scores, P = 2 B for O
    constexpr int kRows = 256, T = D / 16, B = D / 32, P = 2 * B;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint2* const tables = reinterpret_cast<uint2*>(smem);
    uint8_t* const k_lds = smem + kScaleTableBytes;
    uint8_t* const v_lds = k_lds + 2 * Tile::kTile;
    uint32_t* const flags = reinterpret_cast<uint32_t*>(smem + Tile::kFlags);

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit16 = wave & 3;  // which 16 keys of a tile it decodes
    Item it;
    if (!item_of<kRows, false>(p, it)) return;
    const int b = __builtin_amdgcn_readfirstlane(it.b);
    const int head = __builtin_amdgcn_readfirstlane(it.head);
    const int row_tile = __builtin_amdgcn_readfirstlane(it.row_tile);
    const int split = __builtin_amdgcn_readfirstlane(it.split);
    const int own_splits = __builtin_amdgcn_readfirstlane(it.splits);

    const Sequence s = sequence_of(p, b);
    const int row0 = row_tile * kRows, rows = s.tile_rows(p);
    if (p.splits > 1 && split == 0 && row_tile == 0) mark_unowned(p, s, b, head);
    if (row0 >= rows) return;
    const uint32_t four = opaque_four(p);
    const int last_row = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
    const int pos_lo = s.pos0 + (int)p.group.into(row0), pos_hi = s.pos0 + (int)p.group.into(last_row);
    const KeyUnits units = key_units(p, s.len, pos_lo, pos_hi, 64);
    const WholeSteps whole(p, s.len, pos_lo, pos_hi, 32);
    const int per = units_per_split(p, units.n);
    const int begin = split * per;
    const int end = begin + per < units.n ? begin + per : units.n;
    if (split == 0)
        for (int i = own_splits; i < p.splits; i++) mark_empty(p, s.first_row, head, row0, last_row, i);
    if (p.splits > 1 && begin >= end) {
        mark_empty(p, s.first_row, head, row0, last_row, split);
        return;
    }
    uint32_t poisoned = 0;  // groups of O that are NaN
    f32x16 o[B], x;
#pragma unroll
    for (int d = 0; d < B; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0.0f;

    // this lane's codes of the 16 keys that its wave decodes
    const int kq = lane >> 4, vq = (kq & 1) * 2 + (kq >> 1);
    const uint32_t code_at = (lane & 15) * (D / 2) + (kLate ? kq : vq) * (D / 8);
    const uint32_t scale_at = kLate ? (lane & 15) * (D / 16) + kq * (D / 64)
                                   : (lane & 15) * D / 256 * 16 + vq * 4;
    const uint8_t* const codes = kLate ? p.k_codes : p.v_codes;
    const uint8_t* const scales = kLate ? p.k_scales : p.v_scales;
    uint8_t* const k_to = k_lds + ((unit16 >> 1) * T + kq * (D / 64)) * 1024 +
                          (16 * (unit16 & 1) + (lane & 15)) * 16;
    uint8_t* const v_to =
        v_lds + unit16 * B * 1024 + ((vq & 1) * 32 + (lane & 15)) * 16 + (vq >> 1) * 8;

    struct Codes {
        uint32_t w[D / 32], sc;
    };
    auto load = [&](Codes& c, uint64_t at) KV_INLINE {
        UnitCodes<D>::words(codes + at * (8 * D) + code_at, c.w);
        const uint8_t* src = scales + at * D + scale_at;
        if constexpr (!kLate)
            c.sc = *reinterpret_cast<const uint32_t*>(src);
        else if constexpr (D == 64)
            c.sc = *src;
        else
            c.sc = *reinterpret_cast<const uint16_t*>(src);
    };
    Codes now;
    bool bad = false;  // a NaN among the scales of `now` (V)
    auto ref = [&](int i) KV_INLINE {
        return tile_ref(p, s, 4 * units(i < end ? i : end - 1) + unit16);
    };
    // q and the first tiles' codes are asked for together
    typedef TileQ<D, kRows, kPairThreads> QTile;
    typename QTile::Words q_words;
    QTile::ask(p, s, head, row0, rows, tid, q_words);
    __builtin_amdgcn_sched_barrier(0);
    Codes first[3];
    if (begin < end) {
        TileRef r[3];
#pragma unroll
        for (int i = 0; i < 3; i++) r[i] = ref(begin + i);
#pragma unroll
        for (int i = 0; i < (kLate ? 3 : 2); i++) load(first[i], cache_tile(p, head, r[i]));
    }
    fill_scale_tables(tables, tid, kPairThreads);
    half8 q[T];
    float factor, m = kLowest, l = 0.0f;
    int pos;
    QTile::put(k_lds, tid, q_words);
    __syncthreads();
    QTile::take(p, k_lds, 32 * wave + (lane & 31), half, q, factor);
    pos = position_of(p, s, row0 + 32 * wave + (lane & 31), rows);
    now = first[0];

    // The scales of the codes in `now`, looked up one phase before their decode.
    GroupScale look[4];
    auto look_up = [&]() KV_INLINE {
        if constexpr (kLate) {
#pragma unroll
            for (int i = 0; i < D / 64; i++) look[i] = k_scale(tables, (now.sc >> (8 * i)) & 0xFFu);
        } else {
            VPiece<D>::look_up(tables, now.sc, look);
            bad = __builtin_amdgcn_ballot_w64(nan_bytes(now.sc) != 0) != 0;
        }
    };
    // Decode of `now` (one 16-token tile), in T + P slices that go between the
    // products of an A phase: the bits first, then operand by operand.
    KGroup kg[D / 64];
    uint4 operand;
    VPiece<D> vp;
    auto decode = [&](int buf, auto slice_c) KV_INLINE {
        constexpr int n = decltype(slice_c)::value;
        if constexpr (n < T) {
            constexpr int g = n / 4, k = n % 4;
            if constexpr (kLate && k < 3)
                kg[g].template unpack_stage<k>(now.w[2 * g], now.w[2 * g + 1], look[g], four);
            if constexpr (!kLate && k < 3) vp.template unpack_stage<g, k>(now.w, look, four);
            if constexpr (!kLate && n == 0)
                flags[buf * kWaves + unit16] = bad;  // (every lane the same)
        } else if constexpr (!kLate) {
            constexpr int d = n - T;
            uint8_t* const to = v_to + buf * Tile::kTile + (d >> 1) * 1024 + (d & 1) * 256;
            *reinterpret_cast<uint2*>(to) =
                make_uint2(vp.template pair<d, 0>(), vp.template pair<d, 1>());
        } else {
            constexpr int i = (n - T) / 2;  // operand of 8 elements, in two halves
            if constexpr ((n - T) % 2 == 0) {
                operand.x = kg[i / 2].template pair<i % 2, 0>();
                operand.y = kg[i / 2].template pair<i % 2, 1>();
            } else {
                operand.z = kg[i / 2].template pair<i % 2, 2>();
                operand.w = kg[i / 2].template pair<i % 2, 3>();
                *reinterpret_cast<uint4*>(k_to + buf * Tile::kTile + (i / 2) * 1024 +
                                          (i % 2) * 512) = operand;
            }
        }
    };
    half8 ka[P];  // K's operands, P ahead
    auto read_k = [&](int buf, int kb, int t) KV_INLINE {
        return *reinterpret_cast<const half8*>(k_lds + buf * Tile::kTile + (kb * T + t) * 1024 +
                                               lane * 16);
    };
    uint4 prob[2];
    // Largest score of this lane, in parts that go between products.
    float part[6], top;
    auto largest_part = [&](auto part_c) KV_INLINE {
        constexpr int j = decltype(part_c)::value;
        if constexpr (j < 3) {
#pragma unroll
            for (int i = 2 * j; i < 2 * j + 2 && i < 5; i++)
                part[i] = __builtin_fmaxf(__builtin_fmaxf(x[3 * i], x[3 * i + 1]), x[3 * i + 2]);
        } else if constexpr (j == 3) {
            part[5] = __builtin_fmaxf(__builtin_fmaxf(part[0], part[1]), x[15]);
            part[2] = __builtin_fmaxf(__builtin_fmaxf(part[2], part[3]), part[4]);
        } else {
            top = __builtin_fmaxf(part[2], part[5]) * factor;
        }
    };
    // The products of an A phase: scores of the step whose first P operands of K
    // are in ka, then V's operands of keys 32 kb .. of a tile times the
    // probabilities.  Beside each product one operand is asked for,
    // P products ahead of its use: the rest of K, V, the first of the next
    // step's K (tile buffer k_buf, half k_half).  The largest score is taken once
    // the scores are there; f(slice) is the work that goes behind each product.
    auto products = [&](int buf, int kb, int k_buf, int k_half, auto&& f) KV_INLINE {
        const uint8_t* src = v_lds + buf * Tile::kTile + 2 * kb * B * 1024 + lane * 16;
        half8 va[P];
        each<T>([&](auto t_c) KV_INLINE {
            constexpr int t = decltype(t_c)::value;
            if constexpr (t == 0) {
                f32x16 zero;
#pragma unroll
                for (int i = 0; i < 16; i++) zero[i] = 0.0f;
                x = __builtin_amdgcn_mfma_f32_32x32x16_f16(ka[0], q[0], zero, 0, 0, 0);
            } else {
                x = __builtin_amdgcn_mfma_f32_32x32x16_f16(ka[t % P], q[t], x, 0, 0, 0);
            }
            if constexpr (t < T - P)  // the same step's, the other half of this tile or the next's
                ka[t] = read_k(kb == 0 ? buf : k_buf, 1 - kb, t + P);
            else
                va[t - (T - P)] = *reinterpret_cast<const half8*>(src + (t - (T - P)) * 1024);
            f(t_c);
            __builtin_amdgcn_sched_barrier(0);
        });
        each<P>([&](auto n_c) KV_INLINE {
            constexpr int n = decltype(n_c)::value;
            o[n % B] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                va[n], __builtin_bit_cast(half8, prob[n / B]), o[n % B], 0, 0, 0);
            ka[n] = read_k(k_buf, k_half, n);
            f(std::integral_constant<int, T + n>{});
            if constexpr (P == 8 && n >= 3) {
                largest_part(std::integral_constant<int, n - 3>{});
            } else if constexpr (P == 4 && n == 2) {
                each<3>(largest_part);
            } else if constexpr (P == 4 && n == 3) {
                largest_part(std::integral_constant<int, 3>{});
                largest_part(std::integral_constant<int, 4>{});
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // NaN values of V (decoded as zeros) of a 64-key tile: the groups that turn
    // NaN in the rows that see them
    auto poison = [&](int u) KV_INLINE {
#pragma unroll 1
        for (int j = 0; j < 4 * T; j++) {  // 16-token tile j / T, group j % T (T = D / 16)
            const uint64_t at = cache_tile(p, head, tile_ref(p, s, 4 * u + j / T));
            const uint8_t* src = p.v_scales + at * D + (j % T) * 16;
#pragma unroll 1
            for (int t = 0; t < 16; t++) {
                const int key = 64 * u + 16 * (j / T) + t;
                const bool hit = (src[t] & 0x7F) == 0x7F && sees(p, s.len, pos, key);
                poisoned |= (uint32_t)hit << (j % T);
            }
        }
    };

    // What few steps need, behind one branch: keys that some row does not see
    // are hidden, m is raised where a score exceeds it by more than the slack,
    // and NaN values of V are noted.
    auto settle = [&](int key0, uint32_t nan_tile, int u) KV_INLINE {
        const bool all = whole(key0);
        if (all & (__builtin_amdgcn_ballot_w64((top > m + kSlack) | (nan_tile != 0)) == 0)) return;
        if (nan_tile != 0) poison(u);
        if (!all) {
            hide(p, s.len, pos, key0 + 4 * half, x);
            each<5>(largest_part);
        }
        if (__builtin_amdgcn_ballot_w64(top > m + kSlack) == 0) return;
        const float raised = __builtin_fmaxf(top, m);
        const float both = __builtin_fmaxf(raised, __shfl_xor(raised, 32));
        const float alpha = __builtin_amdgcn_exp2f(m - both);
        m = both;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < B; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) o[d][i] *= alpha;
    };
    lds_barrier();
    if (begin < end) {
        // K of tiles 0 and 1, V of tile 0, probabilities of step 0
        const auto decode_tile = [&](int buf) KV_INLINE {
            look_up();
            each<T + P>([&](auto n) KV_INLINE { decode(buf, n); });
        };
        // (a loop: its code is not in the caches yet)
#pragma unroll 1
        for (int t = 0; t < (kLate ? 2 : 1); t++) {
            decode_tile(t);
            now = first[1];
            first[1] = first[2];
        }
        // the tile whose codes are loaded next.  (Its page is asked for in a B phase:
        // a scalar load in flight turns every wait for LDS into one for all of it.)
        constexpr int ahead = kLate ? 3 : 2;
        TileRef next = ref(begin + ahead);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < 16; i++) x[i] = 0.0f;
#pragma unroll
        for (int t = 0; t < T; t++)
            x = __builtin_amdgcn_mfma_f32_32x32x16_f16(read_k(0, 0, t), q[t], x, 0, 0, 0);
        each<5>(largest_part);
        settle(64 * units(begin), 0, 0);
        probabilities(x, factor, m, l, prob);
#pragma unroll
        for (int n = 0; n < P; n++) ka[n] = read_k(0, 1, n);
        if constexpr (!kLate) look_up();
        if constexpr (kLate) lds_barrier();
#pragma unroll 1
        for (int i = begin; i < end; i++) {
            const int buf = (i - begin) & 1, u = units(i);
            const uint32_t at = cache_tile(p, head, next);
            // A(2c), B(2c)
            uint4 f;
            uint32_t nan_tile;
            __builtin_amdgcn_s_setprio(1);
            products(buf, 0, buf ^ 1, 0, [&](auto n) KV_INLINE {
                if constexpr (decltype(n)::value == 0)
                    f = *reinterpret_cast<const uint4*>(flags + buf * kWaves);
                if constexpr (decltype(n)::value == 2) nan_tile = (f.x | f.y) | (f.z | f.w);
                if constexpr (!kLate) decode(buf ^ 1, n);
                if constexpr (!kLate && decltype(n)::value == T) load(now, at);
            });
            __builtin_amdgcn_s_setprio(0);
            lds_barrier();
            settle(64 * u + 32, nan_tile, u);
            next = ref(i + 1 + ahead);
            probabilities(x, factor, m, l, prob);
            if constexpr (kLate) look_up();
            lds_barrier();
            // A(2c + 1), B(2c + 1)
            __builtin_amdgcn_s_setprio(1);
            products(buf, 1, buf ^ 1, 1, [&](auto n) KV_INLINE {
                if constexpr (kLate) decode(buf, n);
                if constexpr (kLate && decltype(n)::value == T) load(now, at);
            });
            __builtin_amdgcn_s_setprio(0);
            lds_barrier();
            settle(i + 1 < end ? 64 * units(i + 1) : kHidden, 0, 0);
            probabilities(x, factor, m, l, prob);
            if constexpr (!kLate) look_up();
            lds_barrier();
        }
        if constexpr (!kLate) lds_barrier();
    }

    // (the row's place from a lane number that the compiler takes for another one:
    // kept across the loop it would cost registers)
    int lane_again = lane;
    asm volatile("" : "+v"(lane_again));
    store_row<D, B>(p, s, head, row0 + 32 * wave + (lane_again & 31), rows, lane_again >> 5, split,
                    0, o, m, l, poisoned);
}

template <int D>
__global__ void __launch_bounds__(kPairThreads, D == 64 ? 4 : 2) prompt_kernel(const Args p) {
    if (threadIdx.x >= kPairThreads / 2)
        prompt_rows<D, true>(p);
    else
        prompt_rows<D, false>(p);
}

// ---------------------------------------------------------------------------
// Wide heads (D = 256, more than 32 rows): tiles of 128 rows, 8 waves.
//
// Here the registers of one wave do not hold Q, O and the operands in flight, so
// two waves of a SIMD, w and w + 4, share 32 rows: each has half of O's dims (the
// words of 8 dims of every V piece that have its number) and computes the
// scores and probabilities of half of the keys, waves 0-3 those of the even steps
// of 32, waves 4-7 those of the odd ones.  Probabilities pass through LDS as they
// are, operands of O's products, and so does the running maximum m, which both
// use: it is read, raised if need be and written by one wave of the two at a time.
// Raised are whole powers of two, so that probabilities that are still to be used are
// scaled exactly as far as fp16 holds them (down to 2^-14 of the largest one, in steps of
// 2^-24 below), and rounded down, so that the largest is at least 1.
//
// As in prompt_rows one wave issues products (A: 16 of its next scores, 16 of O)
// while the other does the VALU work of its step (B).  With c = 64-key tile:
//   phase 2c      waves 0-3: A(c): scores 2c + 2, O += P(2c - 1) V, P(2c) V
//                 waves 4-7: B(c): P(2c + 1)
//   phase 2c + 1  waves 0-3: B(c + 1): P(2c + 2)
//                 waves 4-7: A(c): scores 2c + 3, O += P(2c) V, P(2c + 1) V
// and waves 0-3 add the last odd step's P V after the loop.
//   * waves 0-3 decode K of tile c + 2 in A(c), phase 2c.  K of tile c, in the same
//     buffer, was last read in A(c - 1) of waves 4-7, phase 2c - 1; K of tile c + 2
//     is first read (its first operands, in a B phase) in phase 2c + 1.
//   * waves 4-7 decode V of tile c + 1 in A(c), phase 2c + 1.  V of tile c - 1 was
//     last read in A(c) of waves 0-3, phase 2c; V of tile c + 1 is first read in
//     phase 2c + 2.  So are the NaN flags of a tile, last read in phase 2c + 1.
//   * a pair's probabilities and m are written in the B phases, which take turns,
//     and read by the other wave in its next one, before it writes.
// (Two workgroups per 256 rows that take half of O's dims each and both compute
// all scores took 1.5 times the products and twice the softmax.)
//
// 2048 new of 16384 tokens, 32 heads: 995 to 1010 us, 1020 to 1036 TFLOP/s (the two
// workgroups: 727).  Bound as prompt_rows is, with more decode per product, 128 rows sharing it
// instead of 256.
struct WideTile {
    static constexpr int D = 256, kRows = 128, kTile = 64 * D * 2;
    static constexpr int kProb = kScaleTableBytes + 4 * kTile;  // [4 pairs][2][64 lanes][16]
    static constexpr int kMax = kProb + 4 * 2048;               // [4 pairs][32 rows]
    static constexpr int kFlags = kMax + 4 * 128;
    static constexpr int kLds = kFlags + 2 * kWaves * 4;
};

template <bool kLate>
__device__ __forceinline__ void wide_rows(const Args& p) {
    typedef WideTile Tile;
    constexpr int D = Tile::D, kRows = Tile::kRows, T = D / 16, B = 4, P = 8;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint2* const tables = reinterpret_cast<uint2*>(smem);
    uint8_t* const k_lds = smem + kScaleTableBytes;
    uint8_t* const v_lds = k_lds + 2 * Tile::kTile;
    uint32_t* const flags = reinterpret_cast<uint32_t*>(smem + Tile::kFlags);

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    // which 32 rows, and which 16 keys of a tile it decodes
    const int pair = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
    Item it;
    if (!item_of<kRows, true>(p, it)) return;
    const int b = __builtin_amdgcn_readfirstlane(it.b);
    const int head = __builtin_amdgcn_readfirstlane(it.head);
    const int row_tile = __builtin_amdgcn_readfirstlane(it.row_tile);
    const int split = __builtin_amdgcn_readfirstlane(it.split);
    const int own_splits = __builtin_amdgcn_readfirstlane(it.splits);

    const Sequence s = sequence_of(p, b);
    const int row0 = row_tile * kRows, rows = s.tile_rows(p);
    if (p.splits > 1 && split == 0 && row_tile == 0) mark_unowned(p, s, b, head);
    if (row0 >= rows) return;
    const uint32_t four = opaque_four(p);
    const int last_row = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
    const int pos_lo = s.pos0 + (int)p.group.into(row0), pos_hi = s.pos0 + (int)p.group.into(last_row);
    const KeyUnits units = key_units(p, s.len, pos_lo, pos_hi, 64);
    const WholeSteps whole(p, s.len, pos_lo, pos_hi, 32);
    const int per = units_per_split(p, units.n);
    const int begin = split * per;
    const int end = begin + per < units.n ? begin + per : units.n;
    if (split == 0)
        for (int i = own_splits; i < p.splits; i++) mark_empty(p, s.first_row, head, row0, last_row, i);
    if (p.splits > 1 && begin >= end) {
        mark_empty(p, s.first_row, head, row0, last_row, split);
        return;
    }
    uint32_t poisoned = 0;  // groups of O that are NaN
    f32x16 o[B], x;
#pragma unroll
    for (int d = 0; d < B; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0.0f;

    // this lane's codes of the 16 keys that its wave decodes
    const int kq = lane >> 4, vq = (kq & 1) * 2 + (kq >> 1);
    const uint32_t code_at = (lane & 15) * (D / 2) + (kLate ? vq : kq) * (D / 8);
    const uint32_t scale_at = (lane & 15) * (D / 16) + (kLate ? vq : kq) * 4;
    const uint8_t* const codes = kLate ? p.v_codes : p.k_codes;
    const uint8_t* const scales = kLate ? p.v_scales : p.k_scales;
    uint8_t* const to = kLate
        ? v_lds + pair * 8 * 1024 + ((vq & 1) * 32 + (lane & 15)) * 16 + (vq >> 1) * 8
        : k_lds + ((pair >> 1) * T + kq * (D / 64)) * 1024 + (16 * (pair & 1) + (lane & 15)) * 16;

    struct Codes {
        uint32_t w[D / 32], sc;
    };
    auto load = [&](Codes& c, uint64_t at) KV_INLINE {
        UnitCodes<D>::words(codes + at * (8 * D) + code_at, c.w);
        c.sc = *reinterpret_cast<const uint32_t*>(scales + at * D + scale_at);
    };
    auto ref = [&](int i) KV_INLINE {
        return tile_ref(p, s, 4 * units(i < end ? i : end - 1) + pair);
    };
    // q and the first tiles' codes are asked for together
    typedef TileQ<D, kRows, kPairThreads> QTile;
    typename QTile::Words q_words;
    QTile::ask(p, s, head, row0, rows, tid, q_words);
    __builtin_amdgcn_sched_barrier(0);
    Codes now, first[3];
    if (begin < end) {
        TileRef r[3];
#pragma unroll
        for (int i = 0; i < 3; i++) r[i] = ref(begin + i);
#pragma unroll
        for (int i = 0; i < (kLate ? 2 : 3); i++) load(first[i], cache_tile(p, head, r[i]));
    }
    fill_scale_tables(tables, tid, kPairThreads);
    half8 q[T];
    float factor, m = kLowest, l = 0.0f;
    int pos;
    QTile::put(k_lds, tid, q_words);
    __syncthreads();
    QTile::take(p, k_lds, 32 * pair + (lane & 31), half, q, factor);
    pos = position_of(p, s, row0 + 32 * pair + (lane & 31), rows);
    now = first[0];

    // The scales of the codes in `now`, looked up one phase before their decode.
    GroupScale look[4];
    bool bad = false;  // a NaN among them (V)
    auto look_up = [&]() KV_INLINE {
        if constexpr (kLate) {
            VPiece<D>::look_up(tables, now.sc, look);
            bad = __builtin_amdgcn_ballot_w64(nan_bytes(now.sc) != 0) != 0;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) look[i] = k_scale(tables, (now.sc >> (8 * i)) & 0xFFu);
        }
    };
    // Decode of `now` (one 16-token tile), in 32 slices that go between the
    // products of an A phase: K group by group; V's bits first, then its operands.
    // Behind slice kFree its codes are free.
    constexpr int kFree = kLate ? 12 : 26;
    KGroup kg;
    uint4 operand;
    VPiece<D> vp;
    auto decode = [&](int buf, auto slice_c) KV_INLINE {
        constexpr int n = decltype(slice_c)::value;
        if constexpr (!kLate) {
            constexpr int g = n / 8, k = n % 8;
            uint8_t* const dst = to + buf * Tile::kTile + g * 1024;
            if constexpr (k < 3)
                kg.template unpack_stage<k>(now.w[2 * g], now.w[2 * g + 1], look[g], four);
            if constexpr (k == 3 || k == 5) {
                operand.x = kg.template pair<(k - 3) / 2, 0>();
                operand.y = kg.template pair<(k - 3) / 2, 1>();
            }
            if constexpr (k == 4 || k == 6) {
                operand.z = kg.template pair<(k - 4) / 2, 2>();
                operand.w = kg.template pair<(k - 4) / 2, 3>();
                *reinterpret_cast<uint4*>(dst + (k - 4) / 2 * 512) = operand;
            }
        } else if constexpr (n < 12) {
            if constexpr (n == 0) flags[buf * kWaves + pair] = bad;  // (every lane the same)
            vp.template unpack_stage<n / 3, n % 3>(now.w, look, four);
        } else if constexpr (n < 28) {
            constexpr int d = n - 12;
            *reinterpret_cast<uint2*>(to + buf * Tile::kTile + (d >> 1) * 1024 + (d & 1) * 256) =
                make_uint2(vp.template pair<d, 0>(), vp.template pair<d, 1>());
        }
    };
    half8 ring[P];  // operands, P products ahead of their use
    auto read_k = [&](int buf, int t) KV_INLINE {  // of this wave's step of a tile
        return *reinterpret_cast<const half8*>(k_lds + buf * Tile::kTile + (kLate * T + t) * 1024 +
                                               lane * 16);
    };
    // of product n of a step's 8, keys 32 kb .. of a tile
    auto read_v = [&](int buf, int kb, int n) KV_INLINE {
        return *reinterpret_cast<const half8*>(v_lds + buf * Tile::kTile +
                                               ((2 * kb + n / B) * 8 + kLate * B + n % B) * 1024 +
                                               lane * 16);
    };
    uint4 prob[2], theirs[2];  // this wave's step and the other one's before it
#pragma unroll
    for (int i = 0; i < 2; i++) theirs[i] = make_uint4(0u, 0u, 0u, 0u);
    uint4* const prob_lds = reinterpret_cast<uint4*>(smem + Tile::kProb) + pair * 128 + lane;
    float* const max_lds = reinterpret_cast<float*>(smem + Tile::kMax) + pair * 32 + (lane & 31);
    // Largest score of this lane, in parts that go between products.
    float part[6], top;
    auto largest_part = [&](auto part_c) KV_INLINE {
        constexpr int j = decltype(part_c)::value;
        if constexpr (j < 3) {
#pragma unroll
            for (int i = 2 * j; i < 2 * j + 2 && i < 5; i++)
                part[i] = __builtin_fmaxf(__builtin_fmaxf(x[3 * i], x[3 * i + 1]), x[3 * i + 2]);
        } else if constexpr (j == 3) {
            part[5] = __builtin_fmaxf(__builtin_fmaxf(part[0], part[1]), x[15]);
            part[2] = __builtin_fmaxf(__builtin_fmaxf(part[2], part[3]), part[4]);
        } else {
            top = __builtin_fmaxf(part[2], part[5]) * factor;
        }
    };
    // Product n of the 8 of one step's O, with the operand in the ring.
    auto add = [&](const uint4 (&w)[2], auto n_c) KV_INLINE {
        constexpr int n = decltype(n_c)::value;
        o[n % B] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            ring[n], __builtin_bit_cast(half8, w[n / B]), o[n % B], 0, 0, 0);
    };
    // A: the first P operands of K are in the ring; V's of the other wave's step
    // lie in tile buffer `before`, this wave's in `buf`.
    auto products = [&](int buf, int before, auto&& f) KV_INLINE {
        each<T>([&](auto t_c) KV_INLINE {
            constexpr int t = decltype(t_c)::value;
            if constexpr (t == 0) {
                f32x16 zero;
#pragma unroll
                for (int i = 0; i < 16; i++) zero[i] = 0.0f;
                x = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[0], q[0], zero, 0, 0, 0);
            } else {
                x = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[t % P], q[t], x, 0, 0, 0);
            }
            if constexpr (t < T - P)
                ring[t] = read_k(buf ^ 1, t + P);
            else
                ring[t - (T - P)] = read_v(before, 1 - kLate, t - (T - P));
            f(t_c);
            __builtin_amdgcn_sched_barrier(0);
        });
        each<P>([&](auto n_c) KV_INLINE {
            constexpr int n = decltype(n_c)::value;
            add(theirs, n_c);
            ring[n] = read_v(buf, kLate, n);
            f(std::integral_constant<int, T + n>{});
            if constexpr (n >= 3) largest_part(std::integral_constant<int, n - 3>{});
            __builtin_amdgcn_sched_barrier(0);
        });
        each<P>([&](auto n_c) KV_INLINE {
            constexpr int n = decltype(n_c)::value;
            add(prob, n_c);
            f(std::integral_constant<int, T + P + n>{});
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // NaN values of V (decoded as zeros) of a 64-key tile: the groups that turn
    // NaN in the rows that see them
    auto poison = [&](int u) KV_INLINE {
#pragma unroll 1
        for (int j = 0; j < 4 * T; j++) {  // 16-token tile j / T, group j % T (T = D / 16)
            const uint64_t at = cache_tile(p, head, tile_ref(p, s, 4 * u + j / T));
            const uint8_t* src = p.v_scales + at * D + (j % T) * 16;
#pragma unroll 1
            for (int t = 0; t < 16; t++) {
                const int key = 64 * u + 16 * (j / T) + t;
                const bool hit = (src[t] & 0x7F) == 0x7F && sees(p, s.len, pos, key);
                poisoned |= (uint32_t)hit << (j % T);
            }
        }
    };
    // B: the probabilities of the step of 32 keys from key0 on, whose scores are
    // in x.  k_buf: tile buffer of the next scores' K; u: a tile whose V's NaN flags
    // are in v_buf, and not looked at before (tile 0 comes first: `any`); f is called
    // where LDS has answered.
    auto softmax = [&](int key0, int k_buf, bool any, int v_buf, int u, auto&& f) KV_INLINE {
        float shared = m;
        uint32_t nan_tile = 0;
        if (any) {
            shared = *max_lds;
            theirs[0] = prob_lds[0];
            theirs[1] = prob_lds[64];
            const uint4 nan = *reinterpret_cast<const uint4*>(flags + v_buf * kWaves);
            nan_tile = (nan.x | nan.y) | (nan.z | nan.w);
        }
#pragma unroll
        for (int n = 0; n < P; n++) ring[n] = read_k(k_buf, n);
        // What few steps need, behind one branch: keys that some row does not see
        // are hidden, m is raised where a score exceeds it by more than the slack,
        // or follows the other wave's, and NaN values of V are noted.
        const bool all = whole(key0);
        if (!all | (__builtin_amdgcn_ballot_w64((top > shared + kSlack) | (shared != m) |
                                                (nan_tile != 0)) != 0)) {
            if (__builtin_amdgcn_readfirstlane(nan_tile) != 0) poison(u);
            if (!all) {
                hide(p, s.len, pos, key0 + 4 * half, x);
                each<5>(largest_part);
            }
            float next = shared;
            if (__builtin_amdgcn_ballot_w64(top > shared + kSlack) != 0) {
                const float raised = __builtin_fmaxf(top, shared);
                const float both = __builtin_fmaxf(raised, __shfl_xor(raised, 32));
                // (from the lowest m or to an infinite one there is nothing to keep)
                const float by = __builtin_floorf(both - shared);
                next = by < 65536.0f ? shared + by : both;
                const float alpha = __builtin_amdgcn_exp2f(-by);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    uint32_t w[4] = {theirs[i].x, theirs[i].y, theirs[i].z, theirs[i].w};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const half2v h = __builtin_bit_cast(half2v, w[j]);
                        w[j] = pack_half((float)h[0] * alpha, (float)h[1] * alpha);
                    }
                    theirs[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            const float alpha = __builtin_amdgcn_exp2f(m - next);
            m = next;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < B; d++)
#pragma unroll
                for (int i = 0; i < 16; i++) o[d][i] *= alpha;
        }
        f();
        probabilities(x, factor, m, l, prob);
        prob_lds[0] = prob[0];
        prob_lds[64] = prob[1];
        *max_lds = m;
    };
    lds_barrier();
    if (begin < end) {
        const auto decode_tile = [&](int buf) KV_INLINE {
            look_up();
            each<32>([&](auto n) KV_INLINE { decode(buf, n); });
        };
        // (a loop: its code is not in the caches yet)
#pragma unroll 1
        for (int t = 0; t < (kLate ? 1 : 2); t++) {
            decode_tile(t);
            now = first[1];
            first[1] = first[2];
        }
        // the tile whose codes are loaded next.  (Its page is asked for in a B phase
        // behind LDS's last answer: a scalar load in flight turns every wait for LDS
        // into one for all of it.)
        TileRef next = ref(begin + 3);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < 16; i++) x[i] = 0.0f;
#pragma unroll
        for (int t = 0; t < T; t++)
            x = __builtin_amdgcn_mfma_f32_32x32x16_f16(read_k(0, t), q[t], x, 0, 0, 0);
        each<5>(largest_part);
        if constexpr (!kLate) {  // B(0)
            softmax(64 * units(begin), 1, false, 0, 0, [] {});
            look_up();
        }
        lds_barrier();
#pragma unroll 1
        for (int i = begin; i < end; i++) {
            const int buf = (i - begin) & 1, u = units(i);
            if constexpr (kLate) {  // B(c)
                softmax(64 * u + 32, buf ^ 1, true, buf, u, [&]() KV_INLINE { next = ref(i + 2); });
                look_up();
                lds_barrier();
            }
            // A(c); the first one has no step before it, and adds zeros
            const uint32_t at = cache_tile(p, head, next);
            __builtin_amdgcn_s_setprio(1);
            products(buf, kLate || i == begin ? buf : buf ^ 1, [&](auto n) KV_INLINE {
                decode(kLate ? buf ^ 1 : buf, n);
                if constexpr (decltype(n)::value == kFree) load(now, at);
            });
            __builtin_amdgcn_s_setprio(0);
            lds_barrier();
            if constexpr (!kLate) {  // B(c + 1)
                softmax(i + 1 < end ? 64 * units(i + 1) : kHidden, buf, true, buf, u,
                        [&]() KV_INLINE { next = ref(i + 4); });
                look_up();
                lds_barrier();
            }
        }
        if constexpr (!kLate) {
            const int buf = (end - 1 - begin) & 1;
#pragma unroll
            for (int n = 0; n < P; n++) ring[n] = read_v(buf, 1, n);
            each<P>([&](auto n) KV_INLINE { add(theirs, n); });
        }
        // both waves' sums
        float* const sums = reinterpret_cast<float*>(smem + Tile::kProb) + pair * 512 + lane;
        sums[64 * kLate] = l;
        lds_barrier();
        l += sums[64 * !kLate];
    }

    // (the row's place from a lane number that the compiler takes for another one:
    // kept across the loop it would cost registers)
    int lane_again = lane;
    asm volatile("" : "+v"(lane_again));
    store_row<D, B>(p, s, head, row0 + 32 * pair + (lane_again & 31), rows, lane_again >> 5, split,
                    kLate, o, m, l, poisoned);
}

__global__ void __launch_bounds__(kPairThreads, 2) wide_kernel(const Args p) {
    if (threadIdx.x >= kPairThreads / 2)
        wide_rows<true>(p);
    else
        wide_rows<false>(p);
}

// ---------------------------------------------------------------------------
// Joins the splits of one row per workgroup: latency, 3.5 us for 64 rows of 33
// splits, 4.9 for 256 rows of 32.  All waves read every split's m
// and l at once, lane = split mod 64; then D/4 lanes read one split's
// O as 16 bytes each, the workgroup 1024 / D splits side by side, so that the
// whole row is a handful of independent loads.  (One wave per row with a loop
// over the splits took 19 us for 33 splits, nearly all of it waiting.)
constexpr int kMaxSplits = 128;
constexpr int64_t kMaxKeys = (int64_t)1 << 30;  // of a length hint

// Row of q and query head, as one number, of the n-th row of the partial sums; negative: none.
__device__ __forceinline__ int64_t joined_row(const Args& p, int64_t n) {
    if (n >= p.rows_all) return -1;
    if (p.join_tokens == 0) return n;
    const int64_t token = n / p.heads;
    const int b = (int)(token / p.join_tokens), t = (int)(token - (int64_t)b * p.join_tokens);
    const Sequence s = sequence_of(p, b);
    if (t >= s.rows || s.rows * (int)p.group.n > p.upto) return -1;
    return (int64_t)(s.first_row + t) * p.heads + (n - token * p.heads);
}

template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const Args p) {
    constexpr int kLanes = D / 4, kSide = kThreads / kLanes, kRounds = kMaxSplits / kSide;
    __shared__ float weights[kMaxSplits];
    __shared__ __attribute__((aligned(16))) float sums[kThreads * 4];
    const int64_t at = blockIdx.x, place = joined_row(p, at);
    if (place < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, side = tid / kLanes, d = tid % kLanes;
    constexpr int kPer = kMaxSplits / 64;
    f32x2 ml[kPer];
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        const int i = lane + 64 * j;
        ml[j] = *reinterpret_cast<const f32x2*>(
            p.part_ml + 2 * ((i < p.splits ? i : 0) * p.rows_all + at));
    }
    f32x4 part[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; i++) {
        const int split = i * kSide + side;
        if (i * kSide < p.splits)
            part[i] = *reinterpret_cast<const f32x4*>(
                p.part_o + ((split < p.splits ? split : 0) * p.rows_all + at) * D + 4 * d);
    }
    if (__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(ml[0][1]))) < 0.0f)
        return;  // (of split 0: another launch's row, or none's)
    uint64_t used[kPer];
    float top = ml[0][0], sum = 0.0f;
#pragma unroll
    for (int j = 1; j < kPer; j++) top = __builtin_fmaxf(top, ml[j][0]);
#pragma unroll
    for (int i = 1; i < 64; i *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, i));
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        // zero also for splits without keys, whose O is not there
        const bool in = lane + 64 * j < p.splits && ml[j][1] != 0.0f;
        const float w = in ? __builtin_amdgcn_exp2f(ml[j][0] - top) : 0.0f;
        sum += in ? w * ml[j][1] : 0.0f;
        used[j] = __builtin_amdgcn_ballot_w64(in);
        if (tid < 64) weights[lane + 64 * j] = w;
    }
#pragma unroll
    for (int i = 1; i < 64; i *= 2) sum += __shfl_xor(sum, i);
    __syncthreads();
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kRounds; i++) {
        if (i * kSide < p.splits) {
            const int split = i * kSide + side;
            const float f = weights[split];
            const bool in = used[i * kSide / 64] >> (split & 63) & 1;
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc[j] = in ? __builtin_fmaf(f, part[i][j], acc[j]) : acc[j];
        }
    }
    *reinterpret_cast<f32x4*>(sums + 4 * tid) = acc;
    __syncthreads();
    if (tid < kLanes) {
#pragma unroll
        for (int i = 1; i < kSide; i++) {
            const f32x4 o = *reinterpret_cast<const f32x4*>(sums + 4 * (i * kLanes + tid));
#pragma unroll
            for (int j = 0; j < 4; j++) acc[j] += o[j];
        }
        const float f = sum == 0.0f ? 0.0f : p.v_mul / sum;
        const int64_t row = place / p.heads, hd = place - row * p.heads;
        *reinterpret_cast<uint2*>(p.out + row * p.o_st + hd * p.o_sh + 4 * tid) =
            make_uint2(pack_bf16(acc[0] * f, acc[1] * f), pack_bf16(acc[2] * f, acc[3] * f));
    }
}

// The same for at most kFewSplits splits: one wave per row, no LDS (4096 rows of 6
// splits at D = 128: 5.7 us against 9 a workgroup per row).
constexpr int kFewSplits = 8;

template <int D>
__global__ void __launch_bounds__(kThreads) join_few_kernel(const Args p) {
    constexpr int kLanes = D / 4, kSide = 64 / kLanes, kRounds = kFewSplits / kSide;
    const int64_t at = (int64_t)blockIdx.x * kWaves +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6),
                  place = joined_row(p, at);
    const int lane = threadIdx.x & 63, side = lane / kLanes, d = lane % kLanes;
    if (place < 0) return;
    f32x2 ml[kFewSplits];
#pragma unroll
    for (int i = 0; i < kFewSplits; i++)
        ml[i] = *reinterpret_cast<const f32x2*>(
            p.part_ml + 2 * ((i < p.splits ? i : 0) * p.rows_all + at));
    f32x4 part[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; i++) {
        const int split = i * kSide + side;
        if (i * kSide < p.splits)
            part[i] = *reinterpret_cast<const f32x4*>(
                p.part_o + ((split < p.splits ? split : 0) * p.rows_all + at) * D + 4 * d);
    }
    if (ml[0][1] < 0.0f) return;  // another launch's row, or none's
    float top = ml[0][0], sum = 0.0f;
#pragma unroll
    for (int i = 1; i < kFewSplits; i++) top = __builtin_fmaxf(top, ml[i][0]);
    float w[kFewSplits];
#pragma unroll
    for (int i = 0; i < kFewSplits; i++) {
        // zero also for splits without keys, whose O is not there
        const bool in = i < p.splits && ml[i][1] != 0.0f;
        w[i] = in ? __builtin_amdgcn_exp2f(ml[i][0] - top) : 0.0f;
        sum += in ? w[i] * ml[i][1] : 0.0f;
        ml[i][1] = in ? 1.0f : 0.0f;
    }
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kRounds; i++) {
        if (i * kSide < p.splits) {
            float f = w[i * kSide], in = ml[i * kSide][1];
#pragma unroll
            for (int j = 1; j < kSide; j++) {
                f = side == j ? w[i * kSide + j] : f;
                in = side == j ? ml[i * kSide + j][1] : in;
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc[j] = in != 0.0f ? __builtin_fmaf(f, part[i][j], acc[j]) : acc[j];
        }
    }
#pragma unroll
    for (int i = kLanes; i < 64; i *= 2)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[j] += __shfl_xor(acc[j], i);
    if (side == 0) {
        const float f = sum == 0.0f ? 0.0f : p.v_mul / sum;
        const int64_t row = place / p.heads, hd = place - row * p.heads;
        *reinterpret_cast<uint2*>(p.out + row * p.o_st + hd * p.o_sh + 4 * d) =
            make_uint2(pack_bf16(acc[0] * f, acc[1] * f), pack_bf16(acc[2] * f, acc[3] * f));
    }
}

// ---------------------------------------------------------------------------
// Host side: which kernel, how many splits.
struct Plan {
    enum Kind { kFew, kMany, kPrompt, kWide } kind;
    int blocks;  // row blocks of 16 of a tile (few rows)
    int row_tiles;
    int splits, split_units;
    int64_t items;        // workgroups of a split
    bool compact;
    int above, upto;      // rows of a head of its sequences
    int64_t rows_all;     // of the partial sums
    int64_t ws_o, ws_ml;  // bytes
};

// Rows that the partial sums of a launch have at the most, all splits together: 52 MB of
// them for few rows, 277 MB for the others.  plan_of's rules stay below it: a launch of more than
// one split has no more workgroups than 3 * held (few rows) or 4 * held, each with the rows of
// a tile, and rows that fill less than a whole number of tiles at most twice that.  It
// binds where rows of q are many beside those that the launch is for.
int64_t most_partial_rows(const if4_kv_cache& c, bool few) {
    return (few ? 12582912 : 67108864) / c.head_dim;
}

// Of `batch` sequences with `total_q` tokens together, none with more than `max_q`;
// above: of those with more rows only.  rows_all: of the partial sums.
Plan plan_of(const if4_kv_cache& c, const if4_kv_attention_args& a, int64_t batch, int64_t total_q,
             int64_t max_q, int64_t above, int64_t rows_all) {
    Plan pl;
    pl.above = (int)above;
    pl.upto = INT32_MAX;
    // The kernels by rows of the longest chunk.  Up to 32 rows a wave decodes for
    // its own rows only; beyond, sharing the decode in LDS wins (60 rows of each of
    // 64 heads: 21 us against 28; 64 rows of 16 heads over 16k keys: 40 against
    // 54; 128 rows: 38 against 52).
    const int64_t group = a.heads / c.kv_heads, rows = max_q * group;
    pl.kind = rows <= 32             ? Plan::kFew
              : c.head_dim == 256 ? Plan::kWide
              : rows > 128        ? Plan::kPrompt
                                  : Plan::kMany;
    pl.blocks = rows <= 16 || c.head_dim == 256 ? 1 : 2;
    const int tile = pl.kind == Plan::kFew    ? 16 * pl.blocks
                     : pl.kind == Plan::kPrompt ? 256
                                                : 128;
    pl.row_tiles = (int)((rows + tile - 1) / tile);
    // (at least one, of which a split has at least one unit: kernels divide by its units)
    int64_t keys = a.max_len > 0 ? a.max_len : 1;
    keys = keys < kMaxKeys ? keys : kMaxKeys;
    const int64_t window = a.window < kMaxKeys ? a.window : kMaxKeys;
    const int64_t sinks = a.sinks < kMaxKeys ? a.sinks : kMaxKeys;
    // with a window, what the tokens of one tile see
    const int64_t span = max_q < tile / group + 2 ? max_q : tile / group + 2;
    if (window && window + sinks + span < keys) keys = window + sinks + span;
    // row tiles that hold rows: where chunks differ in length, one of each sequence is
    // half full as a rule
    const bool ragged = total_q < batch * max_q;
    int64_t tiles = batch * pl.row_tiles;
    if (ragged) {
        int64_t about = total_q * group / tile + batch / 2;
        about = about > batch ? about : batch;
        tiles = tiles < about ? tiles : about;
    }
    const int64_t base = c.kv_heads * tiles;
    // Splits of the keys: as many as fill a number of workgroups, with at least so
    // many keys each.
    const bool few = pl.kind == Plan::kFew;
    const int64_t unit = few ? kUnit : 64;
    int64_t s = 1;
    const auto fill = [&](int64_t workgroups, int64_t least) {
        const int64_t n = base > 0 ? workgroups / base : 1, most = (keys + least - 1) / least;
        const int64_t t = n < most ? n : most;
        s = s > t ? s : t;
    };
    if (few) {
        // One workgroup per CU down to one unit of each wave (one sequence of 4097 keys:
        // 10 us, whole 39).  Beyond that the join and the partial sums cost more
        // than fuller CUs bring, unless the splits are long: as many workgroups as
        // the chip holds where each has 1024 keys (64 heads, 8 kv heads, D = 128; 128
        // keys each up to three rounds of workgroups before: 32 sequences of 512 keys
        // 16.0 us, so 10.6; 64 of 512 to 1024 26.9, 18.5; 8 of 1000 to 4000 20.3, 17.1; 4 of
        // 100003 to 131071 120, 114).  Where that leaves few splits of each sequence
        // a long one ends late: three rounds of long splits (64 of 3001 to 12289 keys
        // 127 us, so 123).
        const int64_t held = c.head_dim * pl.blocks <= 128 ? 1024 : 512;
        fill(256, kUnit * kWaves);
        fill(512, 512);
        fill(held, 1024);
        if (base >= held / 4) fill(3 * held, 2048);
    } else if (pl.kind == Plan::kMany) {
        // The same with more work per workgroup (32 chunks of 16 tokens over 512 keys, 64
        // heads: 42 us with 512 workgroups of 256 keys, so 23.5; 32 of 10 over 1000 to
        // 4000 106 with 256 workgroups, so 91).
        fill(256, 256);
        fill(512, 512);
    } else {
        // Prompts, whose partial sums are large: the least of rounds * (start of a
        // workgroup + its tiles of 64 keys) + join, in ns as measured (500 tokens, 32
        // heads, D = 256: 40 us in two splits, 30 whole; 512 of 8192 tokens 164 in two,
        // 250 whole).  Where chunks differ in length contexts will, and workgroups that
        // have no keys leave at once: a quarter more than the chip holds is one round (16
        // chunks of 1 to 32 tokens, 500 to 8000 keys, 32 heads, D = 128: 77 us with 256
        // workgroups, 69 with 320, 97 with 384; D = 256, 24 of 1 to 61 tokens, 61 to
        // 5003 keys, 21 heads: 141 whole, 116 in two; 16 of 16 to 64, 500 to 4000 keys,
        // 32 heads: 118 whole, 131 in two).
        const int64_t held = c.head_dim == 64 ? 512 : 256, start = 7000, step = 1800;
        const int64_t n = (keys + 63) / 64, partial = total_q * a.heads * c.head_dim * 8 / 4000;
        int64_t best = INT64_MAX;
        for (int64_t t = 1; t <= kMaxSplits && (t == 1 || (t * 4 <= n && t * base <= 4 * held));
             t++) {
            const int64_t all = ragged ? base * t * 4 / 5 : base * t;
            const int64_t rounds = all > held ? (all + held - 1) / held : 1;
            const int64_t cost = rounds * (start + (n + t - 1) / t * step) +
                                 (t > 1 ? 4000 + t * partial : 0);
            if (cost < best) {
                best = cost;
                s = t;
            }
        }
    }
    s = s > kMaxSplits ? kMaxSplits : s;
    const int64_t most = most_partial_rows(c, few) / rows_all;
    s = s < most ? s : most > 1 ? most : 1;
    const int64_t units = (keys + unit - 1) / unit;
    pl.split_units = (int)((units + s - 1) / s);
    // whole rounds of the waves, and no split that the hint leaves empty
    if (few && s > 1) pl.split_units = (pl.split_units + kWaves - 1) / kWaves * kWaves;
    if (s > 1) s = (units + pl.split_units - 1) / pl.split_units;
    pl.splits = (int)s;
    // Each sequence has at most one tile that is not full.  Counting costs a workgroup's
    // start 1 to 2 us and pays where keys are split or a quarter of the grid would be
    // empty (3 chunks of 700 to 1531 tokens, D = 64, window 1024: 62 us, so 60).
    const int64_t most_tiles = a.total_q * group / tile + a.batch, all_tiles = a.batch * pl.row_tiles;
    pl.compact = pl.kind != Plan::kFew && a.total_q < a.batch * a.max_q &&
                 (above > 0 || s > 1 || most_tiles * 4 < all_tiles * 3);
    pl.items = c.kv_heads * (pl.compact && most_tiles < all_tiles ? most_tiles : all_tiles);
    pl.rows_all = rows_all;
    pl.ws_o = pl.splits > 1 ? pl.splits * rows_all * c.head_dim * 4 : 0;
    pl.ws_ml = pl.splits > 1 ? pl.splits * rows_all * 8 : 0;
    return pl;
}

// The launches of a call: one, or where most sequences bring much less than the longest
// (single tokens beside a long chunk), one for those that fit a tile of few rows and
// one for the rest, each with its own splits, join and rows of partial sums (32 single
// tokens and a chunk of 512 over 4096 keys, 64 heads: 254 us in tiles of 256 rows all, so
// 139; 8 and a chunk of 2048: 329, 230, of which the chunk alone takes 209; with
// partial sums for all rows of q in both launches the latter took a workspace of 479 MB,
// so 4).
struct Launches {
    Plan of[2];
    int n;
    int64_t workspace;
};
Launches launches_of(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    Launches l;
    l.n = 0;
    const int64_t group = a.heads / c.kv_heads;
    const int64_t few = group <= 16 || c.head_dim == 256 ? 16 : 32;
    if (a.max_q * group > 32 && group <= few && a.total_q * 4 < a.batch * a.max_q) {
        l.of[0] = plan_of(c, a, a.batch, a.batch, few / group, 0, a.batch * (few / group) * a.heads);
        l.of[0].upto = (int)few;
        // as if all that is not single tokens came in chunks of the longest
        int64_t rest = (a.total_q - a.batch + a.max_q - 2) / (a.max_q - 1);
        rest = rest < 1 ? 1 : rest > a.batch ? a.batch : rest;
        l.of[1] = plan_of(c, a, rest, rest * a.max_q, a.max_q, few, a.total_q * a.heads);
        l.n = 2;
    } else {
        l.of[0] = plan_of(c, a, a.batch, a.total_q, a.max_q, 0, a.total_q * a.heads);
        l.n = 1;
    }
    l.workspace = 0;
    for (int i = 0; i < l.n; i++) {
        const int64_t need = l.of[i].ws_o + l.of[i].ws_ml;
        l.workspace = l.workspace > need ? l.workspace : need;
    }
    return l;
}

template <int D>
hipError_t launch(void (*kernel)(Args), int threads, int lds, int64_t grid, const Args& p,
                  hipStream_t stream) {
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kernel,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), lds, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t rows = p.rows_all;
    if (rows > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (p.splits <= kFewSplits)
        hipLaunchKernelGGL((join_few_kernel<D>), dim3((unsigned)((rows + kWaves - 1) / kWaves)),
                           dim3(kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((join_kernel<D>), dim3((unsigned)rows), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

template <int D>
hipError_t dispatch(const Args& p, const Plan& pl, hipStream_t stream) {
    if (pl.items > INT32_MAX) return hipErrorInvalidValue;
    const int64_t grid = pl.items * pl.splits;
    if constexpr (D <= 128) {
        if (pl.kind == Plan::kPrompt)
            return launch<D>(prompt_kernel<D>, kPairThreads, PromptTile<D>::kLds, grid, p, stream);
        if (pl.kind == Plan::kMany)
            return launch<D>(many_rows_kernel<D>, kThreads, ManyRows<D>::kLds, grid, p, stream);
        if (pl.blocks == 2)
            return launch<D>(few_rows_kernel<D, 2>, kThreads, FewRows<D, 2>::kLds, grid, p, stream);
    } else if (pl.kind == Plan::kWide) {
        return launch<D>(wide_kernel, kPairThreads, WideTile::kLds, grid, p, stream);
    }
    return launch<D>(few_rows_kernel<D, 1>, kThreads, FewRows<D, 1>::kLds, grid, p, stream);
}

int clamp_int(int64_t v) { return (int)(v > 0x3FFFFFFF ? 0x3FFFFFFF : v); }

}  // namespace

int64_t kv_attention_workspace(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    return launches_of(c, a).workspace;
}

// What plan_of's choices stay within, as a function that grows with each size: splits by the
// keys that one has at the least, rows of the partial sums by the tokens or, in a
// launch of sequences with few rows, by a tile of each.
int64_t kv_attention_workspace_most(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    const int64_t keys = a.max_len < kMaxKeys ? a.max_len : kMaxKeys;
    const int64_t by_keys = (keys + kUnit * kWaves - 1) / (kUnit * kWaves);
    const int64_t splits = by_keys < kMaxSplits ? by_keys : kMaxSplits;
    if (splits <= 1) return 0;
    const auto rows = [&](bool few, int64_t n) {
        const int64_t most = most_partial_rows(c, few);
        return n < most / splits ? n * splits : most;
    };
    const int64_t all = a.total_q * a.heads, tiles = a.batch * c.kv_heads * 32;
    const int64_t few = rows(true, all > tiles ? all : tiles);
    const int64_t many = a.max_q * (a.heads / c.kv_heads) > 32 ? rows(false, all) : 0;
    return (few > many ? few : many) * (c.head_dim * 4 + 8);
}

hipError_t launch_kv_attention(const if4_kv_cache& c, const if4_kv_attention_args& a,
                               void* workspace, hipStream_t stream) {
    Args p;
    p.k_codes = c.k_codes;
    p.k_scales = c.k_scales;
    p.v_codes = c.v_codes;
    p.v_scales = c.v_scales;
    p.q = reinterpret_cast<const uint16_t*>(a.q);
    p.out = reinterpret_cast<uint16_t*>(a.out);
    p.q_st = a.q_stride_token;
    p.q_sh = a.q_stride_head;
    p.o_st = a.out_stride_token;
    p.o_sh = a.out_stride_head;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.q_starts = a.q_starts;
    p.table_stride = c.pages > 0 ? a.table_stride : 0;  // no pages: no keys
    p.part_o = reinterpret_cast<float*>(workspace);
    p.total_q = (int)a.total_q;
    p.max_q = (int)a.max_q;
    p.pages = (int)c.pages;
    p.kv_heads = (int)c.kv_heads;
    p.heads = (int)a.heads;
    p.group = Divisor(a.heads / c.kv_heads);
    p.batch_heads = (int)(a.batch * c.kv_heads);
    p.batch = (int)a.batch;
    p.causal = a.causal != 0;
    p.window = clamp_int(a.window);
    p.sinks = clamp_int(a.sinks);
    p.tiles = Divisor(c.page_size / 16);
    p.q_scale = a.scale * 1.44269504f;
    p.k_exp = c.k_exp + 9;
    p.v_mul = pow2f(c.v_exp + 9);
    const Launches l = launches_of(c, a);
    for (int i = 0; i < l.n; i++) {
        const Plan& pl = l.of[i];
        p.rows_all = pl.rows_all;
        p.part_ml = p.part_o + pl.ws_o / 4;
        p.compact = pl.compact;
        p.row_tiles = pl.row_tiles;
        p.splits = pl.splits;
        p.split_units = pl.split_units;
        p.above = pl.above;
        p.upto = pl.upto;
        p.join_tokens = pl.upto < INT32_MAX ? pl.upto / (int)p.group.n : 0;
        const hipError_t e = c.head_dim == 64    ? dispatch<64>(p, pl, stream)
                             : c.head_dim == 128 ? dispatch<128>(p, pl, stream)
                                                 : dispatch<256>(p, pl, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace if4
