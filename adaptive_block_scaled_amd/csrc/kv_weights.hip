// Attention weights added up per cached token, for gfx950 (definition in
// include/if4_kv_evict.h).
//
// Two passes over the scores S^T = K Q^T, rows of a tile being (token, query head of one kv
// head's group) pairs as in attention.  stats_kernel finds each row's maximum and sum over
// the keys, by key splits; columns_kernel computes the scores again and adds
// exp2(s - max - log2 sum) over the rows of every key, which it owns alone: no atomics, and
// no order that depends on timing.
//
// A lane holds scores of one query row (matrix-core column) and 16 keys, so that a row's
// maximum and sum, and a key's sum over row tiles, stay in registers until the end.
//
// K enters as 7 times its values: FP4's 7 c s' and INT4's 6 q s' have at most 9 bits, which
// fp16 holds, so that nothing is rounded before the fp32 sums (decoded to its own value, an
// INT4 code would be off by up to 2^-11 of it, more than the fp32 results allow).
//
// Few rows (8 of each kv head; 64 sequences of 7600 tokens, 282 MB of K): 67 us and 82, 4.2
// and 3.6 TB/s (the second reads and writes 31 MB of sums too), each pass bound by the decoding
// of 72 bytes a key beside their loads.  Many rows (16384 of each of 8 kv heads over 16384
// keys, heads of 128): 555 us and 605, about 600 cycles of a SIMD for a block of 32 x 32
// scores, whose matrix products take 256, exponentials 256 and other operations 200 that
// partly run beside the products; two waves share a SIMD.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kv_evict_internal.h"
#include "kv_internal.h"
#include "kv_operand.h"
#include "launch_limit.h"

namespace if4 {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Workgroup barrier that orders LDS only (loads from memory stay in flight).
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// f(0), f(1) .. f(n - 1) with constants.
template <int n, int i = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
    if constexpr (i < n) {
        f(std::integral_constant<int, i>{});
        each<n, i + 1>(f);
    }
}

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kUnit = 32;            // keys of a tile
constexpr float kLowest = -3.0e38f;  // running maximum before any key
constexpr float kSlack = 64.0f;      // how far scores may exceed the running maximum
constexpr int kMaxLen = 0x3FFFFF00;  // keys of a sequence
constexpr int kRawBufferFlags = 0x00020000;  // word 3 of a buffer resource for plain bytes

struct Args {
    const uint8_t *k_codes, *k_scales;
    const uint16_t* q;
    int64_t q_st, q_sh;
    const int32_t *page_table, *seq_lens, *q_starts;
    int64_t table_stride;
    if4_kv_mass mass;
    f32x2* stats;  // [splits][rows of q x heads] maximum (in powers of two) and sum
    int64_t stat_rows;
    half8* rows_q;      // many rows: tiles of 32 rows in operand order, see row_tile
    float* row_factor;  // [..][32]
    int64_t row_tiles;  // of one kv head
    float* part_sums;   // many rows: [parts][pairs][key_blocks][keys of a block]
    int key_blocks, parts;
    int total_q, max_q, pages, kv_heads, heads, batch_heads, row_blocks, splits;
    int causal, window, sinks;
    Divisor tiles;  // of 16 tokens in a page
    Divisor group;  // query heads of a kv head
    float q_scale;  // scale * log2(e) / 7
    int k_exp;      // E of K plus the 12 of its operands
};

struct Sequence {
    int first_row, rows;  // rows of q
    int used;             // the first max_q of them
    int len, pos0;        // keys, position of the first row
    const int32_t* table;
    int64_t mass_row;
    bool there;
};

__device__ __forceinline__ Sequence sequence_of(const Args& p, int b) {
    Sequence s;
    int q0 = p.q_starts[b], q1 = p.q_starts[b + 1];
    q0 = q0 < 0 ? 0 : q0 > p.total_q ? p.total_q : q0;
    q1 = q1 < q0 ? q0 : q1 > p.total_q ? p.total_q : q1;
    s.first_row = q0;
    s.rows = q1 - q0;
    s.used = s.rows < p.max_q ? s.rows : p.max_q;
    int64_t room = p.table_stride * p.tiles.n * 16;
    room = room < kMaxLen ? room : kMaxLen;
    const int64_t len = p.seq_lens[b];
    s.len = (int)(len < 0 ? 0 : len > room ? room : len);
    s.pos0 = s.len - s.rows;
    s.table = p.page_table + b * p.table_stride;
    s.mass_row = p.mass.rows ? p.mass.rows[b] : b;
    s.there = s.rows > 0 && s.mass_row >= 0 && s.mass_row < p.mass.mass_rows;
    return s;
}

// Row of the cache (token of one kv head) that holds key j; j past the last key gives a
// row of the last tile.
__device__ __forceinline__ int64_t cache_row(const Args& p, const Sequence& s, int head, int j) {
    const int last = s.len > 0 ? (s.len - 1) >> 4 : 0;
    const uint32_t t = (uint32_t)((j >> 4) < last ? j >> 4 : last), i = p.tiles.into(t);
    int page = s.table[i];
    page = page < p.pages - 1 ? page : p.pages - 1;
    page = page > 0 ? page : 0;
    return ((int64_t)(page * p.kv_heads + head) * p.tiles.n + (t - i * p.tiles.n)) * 16 + (j & 15);
}

// The multipliers of 7 K 2^-12 2^-E, one per scale byte (see GroupScale).
__device__ __forceinline__ void fill_table(uint2* table, int tid) {
    const float sp = __builtin_amdgcn_cvt_scalef32_f32_fp8((uint32_t)tid & 0x7Fu, 1.0f, 0);
    const bool int4 = (tid & 0x80) != 0;
    const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)(sp * (int4 ? 96.0f : 28.0f)));
    table[tid] = make_uint2(h | h << 16, int4 ? 0u : 0x00010001u);
}

// One key's half row: lane l has key l % 32 of a tile, dims D/2 * (l / 32) on.
template <int D>
struct KeyCodes {
    uint32_t w[D / 16];  // 8 codes each
    uint32_t s[D == 256 ? 2 : 1];
    __device__ __forceinline__ void load(const Args& p, int64_t row, int h) {
        const uint8_t* const c = p.k_codes + row * (D / 2) + h * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 64; i++) {
            const uint4 v = reinterpret_cast<const uint4*>(c)[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
        const uint8_t* const b = p.k_scales + row * (D / 16) + h * (D / 32);
        if constexpr (D == 64) {
            s[0] = *reinterpret_cast<const uint16_t*>(b);
        } else if constexpr (D == 128) {
            s[0] = *reinterpret_cast<const uint32_t*>(b);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(b);
            s[0] = v.x, s[1] = v.y;
        }
    }
    __device__ __forceinline__ void decode(const uint2* table, uint32_t four, half8 (&k)[D / 16]) const {
#pragma unroll
        for (int g = 0; g < D / 32; g++) {
            KGroup u;
            u.unpack(w[2 * g], w[2 * g + 1], k_scale(table, (s[g / 4] >> (8 * (g % 4))) & 0xFFu), four);
            k[2 * g] = u.template operand<0>();
            k[2 * g + 1] = u.template operand<1>();
        }
    }
};

// q of tile row r for lane half h, in fp16 after division by the power of two that brings
// the row's largest magnitude into [1, 2); returns the factor of its scores.  A row
// with an infinity or NaN becomes NaN as a whole.
template <int D>
__device__ __forceinline__ float load_q(const Args& p, const Sequence& s, int kv_head, int r, int h,
                                        half8 (&q)[D / 16]) {
    const int token = (int)p.group.into(r), m = r - token * (int)p.group.n;
    const uint16_t* const x = p.q + (s.first_row + token) * p.q_st +
                              (kv_head * (int)p.group.n + m) * p.q_sh + h * (D / 2);
    uint4 v[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; i++) v[i] = reinterpret_cast<const uint4*>(x)[i];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 16; i++) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
            top = top > lo ? top : lo;
            top = top > hi ? top : hi;
        }
    }
    const uint32_t other = (uint32_t)__shfl_xor((int)top, 32);
    top = top > other ? top : other;
    const int e = top == 0 ? 0 : (int)(top >> 7) - 127;
    const float by = top < 0x7F80u ? __builtin_ldexpf(1.0f, -e) : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < D / 16; i++) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            q[i][2 * j] = (_Float16)(__uint_as_float(w[j] << 16) * by);
            q[i][2 * j + 1] = (_Float16)(__uint_as_float(w[j] & 0xFFFF0000u) * by);
        }
    }
    // finite and above zero, so that a hidden key's -inf stays -inf
    const float c = __builtin_ldexpf(p.q_scale, p.k_exp + e);
    return __builtin_fminf(__builtin_fmaxf(c, 1.17549435e-38f), 3.40282347e38f);
}

template <int D>
__device__ __forceinline__ f32x16 scores(const half8 (&k)[D / 16], const half8 (&q)[D / 16]) {
    f32x16 x = {};
#pragma unroll
    for (int t = 0; t < D / 16; t++) x = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[t], q[t], x, 0, 0, 0);
    return x;
}

// Whether rows at positions lo .. hi all see the keys of `tiles` tiles from key `first` on
// (all of them in the window or all of them first tokens: between these two lie hidden keys),
// and whether any of them may see any of keys first .. first + 31.
__device__ __forceinline__ bool all_seen(const Args& p, int len, int lo, int hi, int first, int tiles = 1) {
    const int end = first + tiles * kUnit - 1;
    return end < len && (!p.causal || end <= lo) && (!p.window || first > hi - p.window || end < p.sinks);
}
__device__ __forceinline__ bool any_seen(const Args& p, int len, int lo, int hi, int first) {
    return first < len && (!p.causal || first <= hi) &&
           (!p.window || first + kUnit - 1 > lo - p.window || first < p.sinks);
}

// Scores (or what they are as exponents) of keys that the row at `pos` does not see become
// -inf.  x[i] is that of key first + 4 h + 8 (i / 4) + i % 4.
__device__ __forceinline__ void hide(const Args& p, int len, int pos, int first, f32x16& x) {
    const int last = p.causal && pos < len - 1 ? pos : len - 1;
    const int lo = p.window ? pos - p.window : -1;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int j = first + 8 * (i >> 2) + (i & 3);
        x[i] = j <= last && (j > lo || j < p.sinks) ? x[i] : -__builtin_inff();
    }
}

// The tiles of keys that rows at positions lo .. hi see: the first `sink`, then those from
// `start` on.
struct KeyTiles {
    int sink, start, n;
    __device__ __forceinline__ KeyTiles(const Args& p, int len, int lo, int hi) {
        const int end = p.causal ? (hi + 1 < len ? hi + 1 : len) : len;
        sink = start = n = 0;
        if (end <= 0) return;
        int first = p.window ? lo - p.window + 1 : 0;
        first = first < 0 ? 0 : first;
        start = first / kUnit;
        const int s = p.sinks < first ? p.sinks : first;
        sink = (s + kUnit - 1) / kUnit;
        sink = sink < start ? sink : start;
        n = sink + (end + kUnit - 1) / kUnit - start;
    }
    __device__ __forceinline__ int operator()(int i) const { return i < sink ? i : i - sink + start; }
};

// ---------------------------------------------------------------------------
// Few rows: those of a sequence and kv head fill no more than one tile.  Here rows lie in
// the accumulators' registers and keys in the lanes (S = Q K^T), so that R <= 8 rows take
// 4 of 16 registers through exp2, and a key's sum over rows is its lane's own.  A
// workgroup takes a split of the keys, its waves one tile of 32 each in turn; the page
// table's entry is on its way two tiles ahead, the codes one.

// A lane's key on its way: the page table's entry, then the codes.
template <int D>
struct KeyAhead {
    int page;
    uint32_t tile, rest;
    KeyCodes<D> codes;
    __device__ __forceinline__ void look_up(const Args& p, const Sequence& s, int j) {
        const int last = (s.len - 1) >> 4;
        const uint32_t t = (uint32_t)((j >> 4) < last ? j >> 4 : last), i = p.tiles.into(t);
        page = s.table[i];
        tile = t - i * p.tiles.n;
    }
    __device__ __forceinline__ void load(const Args& p, int head, int lane) {
        int at = page < p.pages - 1 ? page : p.pages - 1;
        at = at > 0 ? at : 0;
        const uint32_t group = (uint32_t)at * (uint32_t)p.kv_heads + (uint32_t)head;
        codes.load(p, (int64_t)((uint64_t)group * p.tiles.n + tile) * 16 + (lane & 15), lane >> 5);
    }
};

// Row of register r for lane half h.
__device__ __forceinline__ int row_of(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// Scores (or what they are as exponents) of key j that its lane's rows do not see become -inf.
template <int R>
__device__ __forceinline__ void hide_rows(const Args& p, const Sequence& s, int rows, int h, int j, float (&x)[R / 2]) {
#pragma unroll
    for (int r = 0; r < R / 2; r++) {
        const int row = row_of(r, h), pos = s.pos0 + (int)p.group.into(row < rows ? row : rows - 1);
        const bool seen = j < s.len && (!p.causal || j <= pos) && (!p.window || j > pos - p.window || j < p.sinks);
        x[r] = seen ? x[r] : -__builtin_inff();
    }
}

// The split and the (sequence, kv head) pair of a workgroup.  A CU gets every 256th workgroup:
// each split's pairs begin further on by the golden section of all, so that one CU's are of
// many sequences, and CUs have as much to do as one another where lengths differ (8 sequences
// of 2000 to 20000 tokens: 48 us without, 43).
struct Work {
    int split, pair;
    __device__ __forceinline__ Work(const Args& p, int index) {
        split = index / p.batch_heads;
        const uint32_t n = (uint32_t)p.batch_heads;
        const uint32_t on = (uint32_t)((uint64_t)((uint32_t)split * 0x9E3779B9u) * n >> 32);
        const uint32_t at = (uint32_t)index - (uint32_t)split * n + on;
        pair = (int)(at < n ? at : at - n);
    }
};

// What both passes over few rows share: the rows' q, and the tiles of keys in turn.
template <int D, int R>
struct FewRows {
    const Args& p;
    Sequence s;
    int head, lane, h, wave, rows, pos_lo, pos_hi;
    uint32_t four;
    half8 q[D / 16];
    float f[R / 2];

    __device__ __forceinline__ FewRows(const Args& args, int bh, uint2* table) : p(args) {
        const int b = bh / p.kv_heads;
        head = bh - b * p.kv_heads;
        s = sequence_of(p, b);
        lane = threadIdx.x & 63;
        h = lane >> 5;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        rows = s.used * (int)p.group.n;
        four = 4u + ((uint32_t)p.total_q >> 31);
        fill_table(table, threadIdx.x);
    }
    __device__ __forceinline__ void load_rows() {
        const int r = lane & 31;
        const float own = load_q<D>(p, s, head, r < rows ? r : rows - 1, h, q);
        spread(own, f);
        pos_lo = s.pos0;
        pos_hi = s.pos0 + s.used - 1;
    }
    // lane r's value into the registers of row r
    __device__ __forceinline__ void spread(float own, float (&to)[R / 2]) const {
#pragma unroll
        for (int r = 0; r < R / 2; r++) to[r] = __shfl(own, row_of(r, h));
    }
    // each(first key, scores, whether all rows see all keys) for the wave's tiles from .. to - 1,
    // in order; tile(t) is the tile's place
    template <class Tile, class Each>
    __device__ __forceinline__ void go(const uint2* table, int from, int to, Tile&& tile, Each&& each) {
        int t = from + wave;
        if (t >= to) return;
        KeyAhead<D> next;
        const int j = lane & 31;
        next.look_up(p, s, tile(t) * kUnit + j);
        next.load(p, head, lane);
        if (t + kWaves < to) next.look_up(p, s, tile(t + kWaves) * kUnit + j);
        for (; t < to; t += kWaves) {
            const int first = tile(t) * kUnit;
            half8 k[D / 16];
            next.codes.decode(table, four, k);
            if (t + kWaves < to) next.load(p, head, lane);
            if (t + 2 * kWaves < to) next.look_up(p, s, tile(t + 2 * kWaves) * kUnit + j);
            const f32x16 all = scores<D>(q, k);
            float x[R / 2];
#pragma unroll
            for (int r = 0; r < R / 2; r++) x[r] = all[r];
            each(first, x, all_seen(p, s.len, pos_lo, pos_hi, first));
        }
    }
    __device__ __forceinline__ void hide(int first, float (&x)[R / 2]) const {
        hide_rows<R>(p, s, rows, h, first + (lane & 31), x);
    }
};

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 2) few_stats_kernel(const Args p) {
    __shared__ uint2 table[256];
    __shared__ f32x2 part[kWaves][R];
    const Work work(p, blockIdx.x);
    FewRows<D, R> few(p, work.pair, table);
    const Sequence& s = few.s;
    if (!s.there) return;
    few.load_rows();
    __syncthreads();
    const KeyTiles tiles(p, s.len, few.pos_lo, few.pos_hi);
    const int share = (tiles.n + p.splits - 1) / p.splits;
    const int from = work.split * share, to = from + share < tiles.n ? from + share : tiles.n;
    float m[R / 2], l[R / 2];
#pragma unroll
    for (int r = 0; r < R / 2; r++) m[r] = kLowest, l[r] = 0.0f;
    few.go(table, from, to, [&](int t) { return tiles(t); }, [&](int first, float (&x)[R / 2], bool whole) {
        if (!whole) few.hide(first, x);
        float y[R / 2], top = -__builtin_inff();
#pragma unroll
        for (int r = 0; r < R / 2; r++) {
            y[r] = __builtin_fmaf(x[r], few.f[r], -m[r]);
            top = __builtin_fmaxf(top, y[r]);
        }
        if (__builtin_amdgcn_ballot_w64(top > kSlack)) {
#pragma unroll
            for (int r = 0; r < R / 2; r++) {
                const float to = y[r] > kSlack ? x[r] * few.f[r] : m[r];
                l[r] *= __builtin_amdgcn_exp2f(m[r] - to);
                m[r] = to;
                y[r] = __builtin_fmaf(x[r], few.f[r], -to);
            }
        }
#pragma unroll
        for (int r = 0; r < R / 2; r++) l[r] += __builtin_amdgcn_exp2f(y[r]);
    });
#pragma unroll
    for (int r = 0; r < R / 2; r++) {
        float top = m[r];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d));
        float sum = l[r] * __builtin_amdgcn_exp2f(m[r] - top);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) sum += __shfl_xor(sum, d);
        if ((few.lane & 31) == 0) part[few.wave][row_of(r, few.h)] = f32x2{top, sum};
    }
    __syncthreads();
    const int r = threadIdx.x;
    if (r >= few.rows) return;
    float top = kLowest, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) top = __builtin_fmaxf(top, part[w][r][0]);
#pragma unroll
    for (int w = 0; w < kWaves; w++) sum += part[w][r][1] * __builtin_amdgcn_exp2f(part[w][r][0] - top);
    const int token = (int)p.group.into(r), mm = r - token * (int)p.group.n;
    p.stats[work.split * p.stat_rows + (int64_t)(s.first_row + token) * p.heads + few.head * (int)p.group.n + mm] =
        f32x2{top, sum};
}

// The exponent that a row's scores are taken from: log2 of its sum over all keys.  A row
// that sees none adds nothing to any key.
__device__ __forceinline__ float log_sum(const Args& p, const Sequence& s, int kv_head, int r) {
    const int token = (int)p.group.into(r), m = r - token * (int)p.group.n;
    const f32x2* at = p.stats + (int64_t)(s.first_row + token) * p.heads + kv_head * (int)p.group.n + m;
    float top = kLowest, sum = 0.0f;
    for (int i = 0; i < p.splits; i++) {
        const f32x2 v = at[i * p.stat_rows];
        const float t = __builtin_fmaxf(top, v[0]);
        sum = sum * __builtin_amdgcn_exp2f(top - t) + v[1] * __builtin_amdgcn_exp2f(v[0] - t);
        top = t;
    }
    return sum == 0.0f ? __builtin_inff() : top + __builtin_amdgcn_logf(sum);
}

// Where a sequence's sums of one kv head are read and written.
struct Sums {
    const float* in;
    float* out;
    int old, width;  // keys that had sums before; keys that have a place
    __device__ __forceinline__ Sums(const Args& p, const Sequence& s, int head) {
        in = p.mass.in + s.mass_row * p.mass.in_stride_row + head * p.mass.in_stride_head;
        out = p.mass.out + s.mass_row * p.mass.out_stride_row + head * p.mass.out_stride_head;
        old = s.pos0 > 0 ? s.pos0 : 0;
        width = p.mass.width < s.len ? (int)p.mass.width : s.len;
    }
};

// The workgroups go through the keys the other way round than those of the first pass did,
// whose last keys are still in the caches.
template <int D, int R>
__global__ void __launch_bounds__(kThreads, 2) few_columns_kernel(const Args p) {
    __shared__ uint2 table[256];
    const Work work(p, gridDim.x - 1 - blockIdx.x);
    FewRows<D, R> few(p, work.pair, table);
    const Sequence& s = few.s;
    if (!s.there) return;
    const Sums sums(p, s, few.head);
    const int tiles = (sums.width + kUnit - 1) / kUnit, share = (tiles + p.splits - 1) / p.splits;
    const int from = work.split * share, to = from + share < tiles ? from + share : tiles;
    if (from >= to) return;
    few.load_rows();
    float log[R / 2];
    const int r = few.lane & 31;
    few.spread(r < few.rows ? log_sum(p, s, few.head, r) : __builtin_inff(), log);
    __syncthreads();
    // tiles that some row sees: the others' sums are only copied, or start at zero
    const KeyTiles seen(p, s.len, few.pos_lo, few.pos_hi);
    const int sink = seen.n > 0 ? seen.sink : 0, start = seen.n > 0 ? seen.start : tiles;
    const auto write = [&](int first, float v) {
        const int key = first + r;
        if (few.h == 0 && key < sums.width) sums.out[key] = key < sums.old ? sums.in[key] + v : v;
    };
    // (hidden as exponents: of a row that is NaN, what it does not see gets nothing all the same)
    const auto add = [&](int first, float (&x)[R / 2], bool whole) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < R / 2; i++) x[i] = __builtin_fmaf(x[i], few.f[i], -log[i]);
        if (!whole) few.hide(first, x);
#pragma unroll
        for (int i = 0; i < R / 2; i++) v += __builtin_amdgcn_exp2f(x[i]);
        write(first, v + __shfl_xor(v, 32));
    };
    const auto same = [](int t) { return t; };
    const int a = from < sink ? (to < sink ? to : sink) : from;  // tiles from .. a are sinks,
    const int z = a < start ? (to < start ? to : start) : a;     // a .. z hidden, z .. to seen
    few.go(table, from, a, same, add);
    for (int t = a + few.wave; t < z; t += kWaves) write(t * kUnit, 0.0f);
    few.go(table, z, to, same, add);
}

// ---------------------------------------------------------------------------
// Many rows.

// Place of a sequence's tile t of 32 rows: sequences follow one another, each from the tile
// after the one that its first row would share, so that none has the same.
__device__ __forceinline__ int64_t row_tile(const Args& p, const Sequence& s, int b, int head, int t) {
    return head * p.row_tiles + ((int64_t)s.first_row * p.group.n >> 5) + b + t;
}

// Blocks (w, i), w < kOuter and i < kInner, i fastest: fetch(w) brings operands for w from
// LDS, beside the last block of the w before; score(w, i) computes a block; f(w, i, x) takes
// its scores, between the matrix products of the next block.
template <int kOuter, int kInner, int kSteps, class Fetch, class Score, class F>
__device__ __forceinline__ void in_turn(Fetch&& fetch, Score&& score, F&& f) {
    constexpr int kBlocks = kOuter * kInner;
    const auto outer = [](auto n) { return std::integral_constant<int, decltype(n)::value / kInner>{}; };
    const auto inner = [](auto n) { return std::integral_constant<int, decltype(n)::value % kInner>{}; };
    const auto first = std::integral_constant<int, 0>{};
    fetch(first);
    if constexpr (kInner == 1 && kOuter > 1) fetch(std::integral_constant<int, 1>{});
    f32x16 x = score(first, first);
    each<kBlocks>([&](auto n) {
        constexpr int next = decltype(n)::value + 1, w = next / kInner + 1;
        if constexpr (next < kBlocks) {
            const auto m = std::integral_constant<int, next>{};
            if constexpr (next % kInner == kInner - 1 && w < kOuter) fetch(std::integral_constant<int, w>{});
            const f32x16 y = score(outer(m), inner(m));
            f(outer(n), inner(n), x);
            x = y;
#pragma unroll
            for (int j = 0; j < kSteps; j++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);            // MFMA
                __builtin_amdgcn_sched_group_barrier(0x400, 16 / kSteps, 0);  // exp2
                __builtin_amdgcn_sched_group_barrier(0x002, 48 / kSteps, 0);  // other VALU
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);            // LDS read
            }
        } else {
            f(outer(n), inner(n), x);
        }
    });
}

// kTiles tiles of 32 rows per wave and a split of the keys that the workgroup's rows see.
// The keys come in groups of four tiles, of which each wave decodes one into LDS, in
// operand order, for all.
template <int D, int kTiles>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2) stats_kernel(const Args p) {
    constexpr int kRows = kWaves * kTiles * 32;
    __shared__ uint2 table[256];
    __shared__ __attribute__((aligned(16))) half8 keys[2][kWaves][D / 16][64];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bh = blockIdx.x % p.batch_heads, rest = blockIdx.x / p.batch_heads;
    const int block = p.row_blocks - 1 - rest % p.row_blocks, split = rest / p.row_blocks;
    const int b = bh / p.kv_heads, head = bh - b * p.kv_heads;
    const Sequence s = sequence_of(p, b);
    const int rows = s.used * (int)p.group.n, row0 = block * kRows;
    if (!s.there || row0 >= rows) return;
    const uint32_t four = 4u + ((uint32_t)p.total_q >> 31);  // not foldable (see HighBytes)
    fill_table(table, tid);
    const int own0 = row0 + wave * kTiles * 32;  // this wave's rows
    const auto row_at = [&](int i) {
        const int r = own0 + 32 * i + (lane & 31);
        return r < rows ? r : rows - 1;
    };
    half8 q[kTiles][D / 16];
    float factor[kTiles], m[kTiles], l[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; i++) {
        factor[i] = load_q<D>(p, s, head, row_at(i), h, q[i]);
        m[i] = kLowest;
        l[i] = 0.0f;
        // the second pass takes them from here
        if (split == 0 && own0 + 32 * i < rows) {
            const int64_t at = row_tile(p, s, b, head, own0 / 32 + i);
#pragma unroll
            for (int t = 0; t < D / 16; t++) p.rows_q[(at * (D / 16) + t) * 64 + lane] = q[i][t];
            if (h == 0) p.row_factor[at * 32 + lane] = factor[i];
        }
    }
    const auto position = [&](int r) { return s.pos0 + (int)p.group.into(r < rows ? r : rows - 1); };
    const int pos_lo = position(own0), pos_hi = position(own0 + kTiles * 32 - 1);
    const KeyTiles tiles(p, s.len, position(row0), position(row0 + kRows - 1));
    const int share = (tiles.n + p.splits - 1) / p.splits;
    const int from = split * share, to = from + share < tiles.n ? from + share : tiles.n;
    // (tiles past the last are the last one again, and not used)
    const auto tile = [&](int t) { return tiles(t < to ? t : to - 1); };
    KeyAhead<D> next;
    if (from < to) {
        next.look_up(p, s, tile(from + wave) * kUnit + (lane & 31));
        next.load(p, head, lane);
        next.look_up(p, s, tile(from + kWaves + wave) * kUnit + (lane & 31));
    }
    __syncthreads();
    // one block's maximum and sum
    const auto add = [&](int i, const f32x16& x) {
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 16; j++) top = __builtin_fmaxf(top, x[j]);
        top *= factor[i];
        if (__builtin_amdgcn_ballot_w64(top > m[i] + kSlack)) {
            const float to = top > m[i] + kSlack ? top : m[i];
            l[i] *= __builtin_amdgcn_exp2f(m[i] - to);
            m[i] = to;
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 16; j++) sum[j & 1] += __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], factor[i], -m[i]));
        l[i] += sum[0] + sum[1];
    };
    int buffer = 0;
    for (int t = from; t < to; t += kWaves) {
        {
            half8 k[D / 16];
            next.codes.decode(table, four, k);
#pragma unroll
            for (int i = 0; i < D / 16; i++) keys[buffer][wave][i][lane] = k[i];
        }
        if (t + kWaves < to) {
            next.load(p, head, lane);
            next.look_up(p, s, tile(t + 2 * kWaves + wave) * kUnit + (lane & 31));
        }
        lds_barrier();
        const int first = tile(t) * kUnit, last = tile(t + kWaves - 1) * kUnit;
        const auto key = [&](int w, int i) { return keys[buffer][w][i][lane]; };
        if (t + kWaves <= to && last - first == (kWaves - 1) * kUnit &&
            all_seen(p, s.len, pos_lo, pos_hi, first, kWaves)) {
            half8 k[2][D / 16];
            in_turn<kWaves, kTiles, D / 16>(
                [&](auto w) {
#pragma unroll
                    for (int j = 0; j < D / 16; j++) k[decltype(w)::value & 1][j] = key(decltype(w)::value, j);
                },
                [&](auto w, auto i) { return scores<D>(k[decltype(w)::value & 1], q[decltype(i)::value]); },
                [&](auto, auto i, const f32x16& x) { add(decltype(i)::value, x); });
        } else {
            for (int w = 0; w < kWaves && t + w < to; w++) {
                const int at = tile(t + w) * kUnit;
                if (!any_seen(p, s.len, pos_lo, pos_hi, at)) continue;
                half8 k[D / 16];
#pragma unroll
                for (int j = 0; j < D / 16; j++) k[j] = key(w, j);
#pragma unroll
                for (int i = 0; i < kTiles; i++) {
                    f32x16 x = scores<D>(k, q[i]);
                    hide(p, s.len, position(own0 + 32 * i + (lane & 31)), at + 4 * h, x);
                    add(i, x);
                }
            }
        }
        buffer ^= 1;
    }
#pragma unroll
    for (int i = 0; i < kTiles; i++) {
        const float om = __shfl_xor(m[i], 32), ol = __shfl_xor(l[i], 32);
        const float top = __builtin_fmaxf(m[i], om);
        const float sum = l[i] * __builtin_amdgcn_exp2f(m[i] - top) + ol * __builtin_amdgcn_exp2f(om - top);
        const int r = own0 + 32 * i + lane;
        if (h == 0 && r < rows) {
            const int token = (int)p.group.into(r), mm = r - token * (int)p.group.n;
            p.stats[split * p.stat_rows + (int64_t)(s.first_row + token) * p.heads + head * (int)p.group.n + mm] =
                f32x2{top, sum};
        }
    }
}

// kTiles tiles of 32 keys per wave, decoded once; the workgroup goes through the rows that
// may see any of its keys, kRowTiles tiles of 32 at a time, which come into LDS in operand
// order while those before are multiplied.  Where blocks of keys are few, a block's rows are
// parted over workgroups, and join_kernel adds the parts in their order.  (Blocks past the
// planned ones, of sequences longer than they were said to be, are not parted.)
template <int D, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) columns_kernel(const Args p) {
    constexpr int kKeys = kWaves * kTiles * kUnit;
    constexpr int kRowTiles = D == 256 ? 2 : 4;
    constexpr int kPieces = kRowTiles * (D / 16) / kWaves;  // 1 KB pieces that a wave brings
    __shared__ uint2 table[256];
    __shared__ float row_factor[2][kRowTiles * 32], row_log[2][kRowTiles * 32];
    extern __shared__ __attribute__((aligned(16))) half8 rows_q[];  // [2][kRowTiles][D / 16][64]
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bh = blockIdx.x % p.batch_heads, rest = blockIdx.x / p.batch_heads;
    const int part = rest / p.key_blocks, block0 = rest - part * p.key_blocks;
    const int b = bh / p.kv_heads, head = bh - b * p.kv_heads;
    const Sequence s = sequence_of(p, b);
    if (!s.there) return;
    const uint32_t four = 4u + ((uint32_t)p.total_q >> 31);
    const int rows = s.used * (int)p.group.n;
    const Sums sums(p, s, head);
    fill_table(table, tid);
    __syncthreads();
    const int64_t stride = (int64_t)p.key_blocks * kKeys;
    for (int64_t key0 = (int64_t)block0 * kKeys; key0 < sums.width; key0 += stride) {
        const bool parted = p.parts > 1 && key0 < stride;
        if (part > 0 && !parted) break;
        const int first = (int)key0 + wave * kTiles * kUnit;
        // rows that may see keys key0 .. key0 + kKeys - 1: from the one at key0, to the last
        // one whose window reaches back
        int lo = 0, hi = rows;
        if (p.causal) {
            const int64_t t = key0 - s.pos0;
            lo = t <= 0 ? 0 : t >= s.used ? rows : (int)t * (int)p.group.n;
        }
        if (p.window && key0 >= p.sinks) {
            const int64_t t = key0 + kKeys - 1 + p.window - s.pos0;  // first token past
            hi = t <= 0 ? 0 : t >= s.used ? rows : (int)t * (int)p.group.n;
        }
        int t0 = lo / 32, tiles = lo < hi ? (hi + 31) / 32 : t0;
        if (parted) {  // whole steps of kRowTiles, so that only a last part has fewer
            const int share = ((tiles - t0 + p.parts - 1) / p.parts + kRowTiles - 1) / kRowTiles * kRowTiles;
            t0 = t0 + part * share < tiles ? t0 + part * share : tiles;
            tiles = t0 + share < tiles ? t0 + share : tiles;
        }
        const half8* const from = p.rows_q + row_tile(p, s, b, head, 0) * (D / 16 * 64);
        const float* const factors = p.row_factor + row_tile(p, s, b, head, 0) * 32;
        float f_next = 0.0f, log_next = 0.0f;
        // (rows past the last one of a tile have an infinite log; tiles past the last are the
        // last one again, and not used)
        const auto fetch = [&](int t, int buffer) {
            // 1 KB pieces, 16 bytes per lane, straight into LDS (scalar addresses but for the lane)
            constexpr int kTileBytes = D / 16 * 1024;
            const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
                (void*)(from + (int64_t)t * (D / 16 * 64)), 0, kRowTiles * kTileBytes, kRawBufferFlags);
#pragma unroll
            for (int i = 0; i < kPieces; i++) {
                const int piece = wave * kPieces + i, w = piece / (D / 16), last = tiles - 1 - t;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (__attribute__((address_space(3))) void*)(rows_q + (buffer * kRowTiles * (D / 16) + piece) * 64),
                    16, lane * 16, (w < last ? w : last) * kTileBytes + piece % (D / 16) * 1024, 0, 0);
            }
            const int r = 32 * t + tid;
            if (tid < kRowTiles * 32) {
                f_next = r < rows ? factors[r] : 1.0f;
                log_next = r < rows ? log_sum(p, s, head, r) : __builtin_inff();
            }
        };
        const auto arrive = [&](int buffer) {
            if (tid < kRowTiles * 32) {
                row_factor[buffer][tid] = f_next;
                row_log[buffer][tid] = log_next;
            }
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0
            __syncthreads();
        };
        if (t0 < tiles) fetch(t0, 0);
        half8 k[kTiles][D / 16];
#pragma unroll
        for (int i = 0; i < kTiles; i++) {
            KeyCodes<D> codes;
            codes.load(p, cache_row(p, s, head, first + i * kUnit + (lane & 31)), h);
            codes.decode(table, four, k[i]);
        }
        float acc[kTiles][16] = {};
        int buffer = 0;
        if (t0 < tiles) arrive(0);
        for (int t = t0; t < tiles; t += kRowTiles) {
            if (t + kRowTiles < tiles) fetch(t + kRowTiles, buffer ^ 1);
            const auto operand = [&](int w, int i) { return rows_q[((buffer * kRowTiles + w) * (D / 16) + i) * 64 + lane]; };
            const auto add = [&](int i, const f32x16& x, float f, float log) {
#pragma unroll
                for (int j = 0; j < 16; j++) acc[i][j] += __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], f, -log));
            };
            const auto position = [&](int r) { return s.pos0 + (int)p.group.into(r < rows ? r : rows - 1); };
            const int pos_lo = position(32 * t), pos_hi = position(32 * (t + kRowTiles) - 1);
            if (all_seen(p, s.len, pos_lo, pos_hi, first, kTiles)) {
                half8 q[2][D / 16];
                float f[2], log[2];
                in_turn<kRowTiles, kTiles, D / 16>(
                    [&](auto w) {
                        constexpr int at = decltype(w)::value;
#pragma unroll
                        for (int j = 0; j < D / 16; j++) q[at & 1][j] = operand(at, j);
                        f[at & 1] = row_factor[buffer][32 * at + (lane & 31)];
                        log[at & 1] = row_log[buffer][32 * at + (lane & 31)];
                    },
                    [&](auto w, auto i) { return scores<D>(k[decltype(i)::value], q[decltype(w)::value & 1]); },
                    [&](auto w, auto i, const f32x16& x) {
                        add(decltype(i)::value, x, f[decltype(w)::value & 1], log[decltype(w)::value & 1]);
                    });
            } else {
                for (int w = 0; w < kRowTiles && t + w < tiles; w++) {
                    const int r0 = 32 * (t + w), lo_w = position(r0), hi_w = position(r0 + 31);
                    half8 q[D / 16];
#pragma unroll
                    for (int i = 0; i < D / 16; i++) q[i] = operand(w, i);
                    const float f = row_factor[buffer][32 * w + (lane & 31)];
                    const float log = row_log[buffer][32 * w + (lane & 31)];
#pragma unroll
                    for (int i = 0; i < kTiles; i++) {
                        const int key = first + i * kUnit;
                        if (!any_seen(p, s.len, lo_w, hi_w, key)) continue;
                        f32x16 x = scores<D>(k[i], q);
                        // (hidden as exponents, as in few_columns_kernel)
#pragma unroll
                        for (int j = 0; j < 16; j++) x[j] = __builtin_fmaf(x[j], f, -log);
                        hide(p, s.len, position(r0 + (lane & 31)), key + 4 * h, x);
#pragma unroll
                        for (int j = 0; j < 16; j++) acc[i][j] += __builtin_amdgcn_exp2f(x[j]);
                    }
                }
            }
            buffer ^= 1;
            if (t + kRowTiles < tiles) arrive(buffer);
        }
        __syncthreads();  // (the next keys' rows come into the same buffers)
#pragma unroll
        for (int i = 0; i < kTiles; i++)
#pragma unroll
            for (int j = 0; j < 16; j++) {
                float v = acc[i][j];
#pragma unroll
                for (int d = 1; d < 32; d *= 2) v += __shfl_xor(v, d);
                const int key = first + i * kUnit + 4 * h + 8 * (j >> 2) + (j & 3);
                if ((lane & 31) == j && key < sums.width) {
                    if (parted)
                        p.part_sums[((int64_t)part * p.batch_heads + bh) * stride + key] = v;
                    else
                        sums.out[key] = key < sums.old ? sums.in[key] + v : v;
                }
            }
    }
}

// The parts' sums of a block of keys, one to a thread, added in their order.
__global__ void join_kernel(const Args p) {
    const int bh = blockIdx.x % p.batch_heads, b = bh / p.kv_heads;
    const int key = blockIdx.x / p.batch_heads * blockDim.x + threadIdx.x;
    const Sequence s = sequence_of(p, b);
    if (!s.there) return;
    const Sums sums(p, s, bh - b * p.kv_heads);
    if (key >= sums.width) return;
    const int64_t stride = (int64_t)p.key_blocks * blockDim.x;
    float v = 0.0f;
    for (int i = 0; i < p.parts; i++) v += p.part_sums[((int64_t)i * p.batch_heads + bh) * stride + key];
    sums.out[key] = key < sums.old ? sums.in[key] + v : v;
}

struct Plan {
    int few;        // rows of a tile where they fill no more than one, else 0
    int row_tiles;  // many: 32-row tiles of a wave of the first pass
    int key_tiles;  // many: 32-key tiles of a wave of the second
    int64_t row_blocks, splits, key_blocks;
    int64_t parts;  // many: of a key block's rows
};

constexpr int kMostSplits = 64;

// Key splits fill the chip: kFull workgroups, four to a CU (a split has two tiles for each of
// its waves at least).  Few rows of so many pairs that fewer than two splits of each would do
// that take twice as many, so that workgroups that are done early have others after them.  In
// us, 1024 workgroups and 2048:  8 sequences of 2000 to 20000 tokens, 8 kv heads, 43, 61;  32
// of 3001 to 12289 88, 95;  4 of 100003 to 131071 137, 169;  64 of 3001 to 12289 158, 157;  100
// of 100 to 9000 160, 153.
constexpr int kFull = 1024;

Plan plan_of(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    Plan p;
    const int64_t rows = a.max_q * (a.heads / c.kv_heads), pairs = a.batch * c.kv_heads;
    const int64_t units = (a.max_len < kMaxLen ? a.max_len : kMaxLen) / kUnit + 1;
    p.few = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 0;
    p.row_tiles = c.head_dim == 256 ? 1 : 2;
    const int64_t block = 32 * kWaves * p.row_tiles;
    p.row_blocks = p.few ? 1 : (rows + block - 1) / block;
    const int64_t groups = pairs * p.row_blocks, full = p.few && 2 * pairs > kFull ? 2 * kFull : kFull;
    const int64_t most = (units + 2 * kWaves - 1) / (2 * kWaves);
    p.splits = groups >= full ? 1 : (full + groups - 1) / groups;
    p.splits = p.splits < most ? p.splits : most;
    p.splits = p.splits < kMostSplits ? p.splits : kMostSplits;
    p.key_tiles = c.head_dim == 256 ? 1 : 2;
    const int64_t keys = kWaves * p.key_tiles;
    p.key_blocks = (units + keys - 1) / keys;
    const int64_t limit = most_groups(kThreads) / pairs;  // (the kernel goes on to what lies past them)
    p.key_blocks = p.key_blocks < limit ? p.key_blocks : limit > 0 ? limit : 1;
    // (a part has 8 tiles of rows at least)
    const int64_t blocks = pairs * p.key_blocks, tiles = (rows + 31) / 32;
    p.parts = p.few || blocks >= kFull / 2 ? 1 : (kFull + blocks - 1) / blocks;
    p.parts = p.parts < tiles / 8 ? p.parts : tiles / 8 > 1 ? tiles / 8 : 1;
    return p;
}

// Sums of the parts, and the most that any call has: fewer than kFull + kFull / 2 workgroups.
int64_t part_bytes(const Plan& p, const if4_kv_cache& c, const if4_kv_attention_args& a) {
    return p.parts > 1 ? p.parts * a.batch * c.kv_heads * p.key_blocks * kWaves * p.key_tiles * kUnit * 4 : 0;
}
constexpr int64_t kMostPartBytes = (int64_t)(kFull + kFull / 2) * kWaves * 2 * kUnit * 4;

template <int D, int R>
hipError_t launch_few(const Args& p, unsigned groups, hipStream_t stream) {
    hipLaunchKernelGGL((few_stats_kernel<D, R>), dim3(groups), dim3(kThreads), 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((few_columns_kernel<D, R>), dim3(groups), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

template <int D, int kRows, int kKeys>
hipError_t launch_many(const Args& p, unsigned groups, unsigned columns, hipStream_t stream) {
    hipLaunchKernelGGL((stats_kernel<D, kRows>), dim3(groups), dim3(kThreads), 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    constexpr int kSmem = 2 * (D == 256 ? 2 : 4) * 32 * D * 2;
    // dynamic LDS above 64 KB (with the static) must be allowed per kernel (idempotent, any device)
    const hipError_t allowed = hipFuncSetAttribute((const void*)columns_kernel<D, kKeys>,
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (allowed != hipSuccess) return allowed;
    hipLaunchKernelGGL((columns_kernel<D, kKeys>), dim3(columns * p.parts), dim3(kThreads), kSmem, stream, p);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess || p.parts == 1) return st;
    hipLaunchKernelGGL(join_kernel, dim3(columns), dim3(kWaves * kKeys * kUnit), 0, stream, p);
    return hipGetLastError();
}

template <int D>
hipError_t launch(const Args& p, const Plan& plan, unsigned groups, unsigned columns, hipStream_t stream) {
    switch (plan.few) {
        case 8: return launch_few<D, 8>(p, groups, stream);
        case 16: return launch_few<D, 16>(p, groups, stream);
        case 32: return launch_few<D, 32>(p, groups, stream);
    }
    if constexpr (D == 256)
        return launch_many<D, 1, 1>(p, groups, columns, stream);
    else
        return launch_many<D, 2, 2>(p, groups, columns, stream);
}

}  // namespace

// Workspace: the splits' maxima and sums, and for many rows q in operand order and the parts' sums.
namespace {
int64_t stat_bytes(int64_t splits, const if4_kv_attention_args& a) {
    return (splits * a.total_q * a.heads * 8 + 15) & ~(int64_t)15;
}
int64_t row_tiles(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    return a.total_q * (a.heads / c.kv_heads) / 32 + a.batch + 1;
}
int64_t row_bytes(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    return row_tiles(c, a) * c.kv_heads * 32 * (2 * c.head_dim + 4);
}
}  // namespace

int64_t kv_weights_workspace(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    const Plan p = plan_of(c, a);
    return stat_bytes(p.splits, a) + (p.few ? 0 : row_bytes(c, a) + part_bytes(p, c, a));
}

// (no call has more splits, nor rows in more tiles, nor more parts)
int64_t kv_weights_workspace_most(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    return stat_bytes(kMostSplits, a) + row_bytes(c, a) + kMostPartBytes;
}

hipError_t launch_kv_weights(const if4_kv_cache& c, const if4_kv_attention_args& a,
                             const if4_kv_mass& m, void* workspace, hipStream_t stream) {
    const Plan plan = plan_of(c, a);
    Args p;
    p.k_codes = c.k_codes;
    p.k_scales = c.k_scales;
    p.q = reinterpret_cast<const uint16_t*>(a.q);
    p.q_st = a.q_stride_token;
    p.q_sh = a.q_stride_head;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.q_starts = a.q_starts;
    p.table_stride = a.table_stride;
    p.mass = m;
    p.stats = reinterpret_cast<f32x2*>(workspace);
    p.stat_rows = a.total_q * a.heads;
    p.row_tiles = row_tiles(c, a);
    p.rows_q = reinterpret_cast<half8*>(reinterpret_cast<uint8_t*>(workspace) + stat_bytes(plan.splits, a));
    p.row_factor = reinterpret_cast<float*>(p.rows_q + p.row_tiles * c.kv_heads * 32 * c.head_dim / 8);
    p.part_sums = p.row_factor + p.row_tiles * c.kv_heads * 32;
    p.key_blocks = (int)plan.key_blocks;
    p.parts = (int)plan.parts;
    p.total_q = (int)a.total_q;
    p.max_q = (int)a.max_q;
    p.pages = (int)c.pages;
    p.kv_heads = (int)c.kv_heads;
    p.heads = (int)a.heads;
    const int64_t pairs = a.batch * c.kv_heads;
    p.batch_heads = (int)pairs;
    p.row_blocks = (int)plan.row_blocks;
    p.splits = (int)plan.splits;
    p.causal = a.causal;
    p.window = (int)(a.window < kMaxLen ? a.window : 0);
    p.sinks = (int)(a.sinks < kMaxLen ? a.sinks : kMaxLen);
    p.tiles = Divisor(c.page_size / 16);
    p.group = Divisor(a.heads / c.kv_heads);
    p.q_scale = a.scale * 1.4426950408889634f / 7.0f;
    p.k_exp = c.k_exp + 12;
    const int64_t stat_groups = pairs * plan.row_blocks * plan.splits;
    if (!launchable(stat_groups, kThreads)) return hipErrorInvalidConfiguration;
    const unsigned groups = (unsigned)stat_groups, columns = (unsigned)(pairs * plan.key_blocks);
    return c.head_dim == 64    ? launch<64>(p, plan, groups, columns, stream)
           : c.head_dim == 128 ? launch<128>(p, plan, groups, columns, stream)
                               : launch<256>(p, plan, groups, columns, stream);
}

}  // namespace if4
