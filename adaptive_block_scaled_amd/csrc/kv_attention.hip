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
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "if4_internal.h"
#include "kv_internal.h"
#include "kv_operand.h"

namespace if4 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kUnit = 32;             // keys that a wave takes at once
constexpr float kLowest = -3.0e38f;   // running maximum before any key
constexpr float kSlack = 8.0f;        // how far scores may exceed it

struct Args {
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_st, q_sh, o_st, o_sh;
    const int32_t *page_table, *seq_lens, *q_starts;
    int64_t table_stride;
    float *part_o, *part_ml;  // splits > 1: [splits][total_q * heads][D], [..][2]
    int64_t rows_all;         // total_q * heads
    int total_q, pages, kv_heads, heads, group, batch_heads, row_tiles, splits;
    int causal, window, sinks;
    // 16-token tiles per page, and its reciprocal: n / d = n * magic >> shift
    uint32_t page_tiles, page_magic;
    int page_shift;
    float q_scale;  // scale * log2(e)
    int k_exp;      // E of K plus the 9 of its operands
    float v_mul;    // 2^(E of V + 9)
};

// One sequence, as a workgroup sees it.
struct Sequence {
    int first_row, rows;  // rows of q
    int len, pos0;        // keys, position of its first row
    const int32_t* table;
};

__device__ __forceinline__ Sequence sequence_of(const Args& p, int b) {
    Sequence s;
    int q0 = p.q_starts[b], q1 = p.q_starts[b + 1];
    q0 = q0 < 0 ? 0 : q0 > p.total_q ? p.total_q : q0;
    q1 = q1 < q0 ? q0 : q1 > p.total_q ? p.total_q : q1;
    s.first_row = q0;
    s.rows = q1 - q0;
    const int64_t room = p.table_stride * p.page_tiles * 16;
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

// Cache tile (16 tokens) of one kv head that holds keys 16 n .. 16 n + 15 of
// a sequence; n past its last key gives some valid tile.
__device__ __forceinline__ int64_t cache_tile(const Args& p, const Sequence& s, int head, int n) {
    const int last = s.len > 0 ? (s.len - 1) >> 4 : 0;
    const uint32_t m = (uint32_t)(n < last ? n : last);
    const uint32_t i = (uint32_t)((uint64_t)m * p.page_magic >> p.page_shift);
    int page = s.table[i];
    page = page < 0 ? 0 : page >= p.pages ? p.pages - 1 : page;
    return ((int64_t)page * p.kv_heads + head) * p.page_tiles + (m - i * p.page_tiles);
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const f32x2 t = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(t, half2v));
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

// Exponent that brings a row whose largest magnitude is a into [1, 2).
__device__ __forceinline__ int row_exponent(float a) {
    const int e = (int)(__float_as_uint(a) >> 23) - 127;
    return a == 0.0f ? 0 : e;
}

// q in fp16, divided by 2^e (exact down to 2^-24 of the row's largest); a row
// with an infinity or NaN has NaN scores, whatever the keys.
__device__ __forceinline__ float q_value(float x, int e) {
    return __builtin_fabsf(x) <= 3.40282347e38f ? __builtin_ldexpf(x, -e)
                                                : __uint_as_float(0x7FC00000u);
}

// ---------------------------------------------------------------------------
// Few rows (a decode step, short chunks): tiles of 16 * kBlocks rows.
//
// Each wave takes its own units of 32 keys, with its own m, l and O, and reads
// their codes straight from memory into operands: v_mfma_f32_16x16x32_f16 of
// K lane l = (key l % 16, quarter l / 16 of D) is a contiguous 1 KB of the
// cache per load at D = 128, and so is V's, lane l = (piece l % 16, tokens
// 4 (l / 16) ..).  Nothing is shared but the scale tables, until the four
// waves' results are joined in LDS.
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
    __device__ __forceinline__ void load(const Args& p, const Sequence& s, int head, int unit,
                                         int lane) {
        const uint32_t code = (lane & 15) * (D / 2) + (lane >> 4) * (D / 8);
        const uint32_t ksc = (lane & 15) * (D / 16) + (lane >> 4) * (D / 64);
        const uint32_t vsc = (lane & 15) * D / 256 * 16 + (lane >> 4) * 4;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int64_t at = cache_tile(p, s, head, 2 * unit + t);
            words(p.k_codes + at * (8 * D) + code, k[t]);
            words(p.v_codes + at * (8 * D) + code, v[t]);
            const uint8_t* kp = p.k_scales + at * D + ksc;
            if constexpr (D == 64)
                ks[t] = *kp;
            else if constexpr (D == 128)
                ks[t] = *reinterpret_cast<const uint16_t*>(kp);
            else
                ks[t] = *reinterpret_cast<const uint32_t*>(kp);
            vs[t] = *reinterpret_cast<const uint32_t*>(p.v_scales + at * D + vsc);
        }
    }
};

template <int D, int kBlocks>
struct FewRows {
    static constexpr int kRows = 16 * kBlocks;
    static constexpr int kPad = D + 4;
    static constexpr int kLds = kScaleTableBytes + kWaves * 16 * kPad * 4 + 2 * kWaves * kRows * 4;
};

template <int D, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks == 1 && D <= 128 ? 3 : 1) few_rows_kernel(const Args p) {
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
    const int row0 = row_tile * kRows, rows = s.rows * p.group;
    if (row0 >= rows) return;
    fill_scale_tables(tables, tid, kThreads);

    const int last_row = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
    const int pos_lo = s.pos0 + row0 / p.group, pos_hi = s.pos0 + last_row / p.group;
    const KeyUnits units = key_units(p, s.len, pos_lo, pos_hi, kUnit);
    const int per = (units.n + p.splits - 1) / p.splits;
    const int begin = split * per;
    const int end = begin + per < units.n ? begin + per : units.n;

    // this lane's row of each block, its q as operands, and what it sees:
    // keys <= see_hi that are > see_lo or < sinks
    half8 q[kBlocks][D / 32];
    float factor[kBlocks];
    int see_hi[kBlocks], see_lo[kBlocks];
#pragma unroll
    for (int nr = 0; nr < kBlocks; nr++) {
        const int r = row0 + 16 * nr + (lane & 15);
        const int rc = r < rows ? r : rows - 1;
        const int t = rc / p.group, g = rc - t * p.group;
        const uint16_t* src = p.q + (s.first_row + t) * p.q_st +
                              (int64_t)(head * p.group + g) * p.q_sh + (lane >> 4) * (D / 4);
        uint4 raw[D / 32];
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; i++) {
            raw[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                a = __builtin_fmaxf(a, __uint_as_float((w[j] << 16) & 0x7FFFFFFFu));
                a = __builtin_fmaxf(a, __uint_as_float(w[j] & 0x7FFF0000u));
            }
        }
        a = __builtin_fmaxf(a, __shfl_xor(a, 16));
        a = __builtin_fmaxf(a, __shfl_xor(a, 32));
        const int e = row_exponent(a);
#pragma unroll
        for (int i = 0; i < D / 32; i++) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            uint4 h;
            uint32_t* hw = &h.x;
#pragma unroll
            for (int j = 0; j < 4; j++)
                hw[j] = pack_half(q_value(__uint_as_float(w[j] << 16), e),
                                  q_value(__uint_as_float(w[j] & 0xFFFF0000u), e));
            q[nr][i] = __builtin_bit_cast(half8, h);
        }
        factor[nr] = score_factor(p, e);
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

    auto compute = [&](const UnitCodes<D>& c, int unit) {
        const int key0 = unit * kUnit;
        f32x4 acc[2][kBlocks];
#pragma unroll
        for (int t = 0; t < 2; t++) {
#pragma unroll
            for (int nr = 0; nr < kBlocks; nr++) acc[t][nr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < D / 32; i++) {
                const GroupScale sc = k_scale(tables, (c.ks[t] >> (8 * (i / 2))) & 0xFFu);
                const half8 a = decode_k_word(c.k[t][i], sc);
#pragma unroll
                for (int nr = 0; nr < kBlocks; nr++)
                    acc[t][nr] =
                        __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[nr][i], acc[t][nr], 0, 0, 0);
            }
        }
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
            top *= factor[nr];
            if (__builtin_amdgcn_ballot_w64(top > m[nr] + kSlack) != 0) {
                top = __builtin_fmaxf(top, m[nr]);
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
            for (int j = 0; j < 8; j++) {
                x[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], factor[nr], -m[nr]));
                l[nr] += x[j];
            }
            prob[nr] = make_uint4(pack_half(x[0], x[1]), pack_half(x[2], x[3]),
                                  pack_half(x[4], x[5]), pack_half(x[6], x[7]));
        }
        uint32_t v0[M][2], v1[M][2];
        decode_v_piece<D>(c.v[0], c.vs[0], tables, v0);
        decode_v_piece<D>(c.v[1], c.vs[1], tables, v1);
#pragma unroll
        for (int d = 0; d < M; d++) {
            const half8 a =
                __builtin_bit_cast(half8, make_uint4(v0[d][0], v0[d][1], v1[d][0], v1[d][1]));
#pragma unroll
            for (int nr = 0; nr < kBlocks; nr++)
                o[d][nr] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    a, __builtin_bit_cast(half8, prob[nr]), o[d][nr], 0, 0, 0);
        }
        // NaN values of V (decoded as zeros): into the rows that see them
        if (__builtin_amdgcn_ballot_w64((nan_bytes(c.vs[0]) | nan_bytes(c.vs[1])) != 0) != 0) {
#pragma unroll 1
            for (int j = 0; j < 8; j++) {
                const uint32_t byte = ((j >> 2 ? c.vs[1] : c.vs[0]) >> (8 * (j & 3))) & 0x7Fu;
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

    // two register sets in turn: the next unit's codes are on their way while
    // one is computed, and no loaded value is copied (that would wait for it)
    int i = begin + wave;
    if (i < end) {
        UnitCodes<D> c0, c1;
        c0.load(p, s, head, units(i), lane);
        while (true) {
            const int n1 = i + kWaves < end ? i + kWaves : i;
            c1.load(p, s, head, units(n1), lane);
            compute(c0, units(i));
            i += kWaves;
            if (i >= end) break;
            const int n2 = i + kWaves < end ? i + kWaves : i;
            c0.load(p, s, head, units(n2), lane);
            compute(c1, units(i));
            i += kWaves;
            if (i >= end) break;
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
            const int t = r / p.group, g = r - t * p.group;
            const int64_t row = s.first_row + t, hd = head * p.group + g;
            if (p.splits == 1) {
                const float f = sum == 0.0f ? 0.0f : p.v_mul / sum;
                uint32_t* dst =
                    reinterpret_cast<uint32_t*>(p.out + row * p.o_st + hd * p.o_sh + (tid & 15) * M);
#pragma unroll
                for (int d = 0; d < M; d += 2) dst[d / 2] = pack_bf16(acc[d] * f, acc[d + 1] * f);
            } else {
                const int64_t at = split * p.rows_all + row * p.heads + hd;
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

// Joins the splits of every row: one wave per row, lane l the dims l D/64 ..
template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const Args p) {
    const int64_t at = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (at >= p.rows_all) return;
    constexpr int E = D / 64;
    float top = kLowest;
    for (int i = 0; i < p.splits; i++)
        top = __builtin_fmaxf(top, p.part_ml[2 * (i * p.rows_all + at)]);
    float sum = 0.0f, acc[E];
#pragma unroll
    for (int d = 0; d < E; d++) acc[d] = 0.0f;
    for (int i = 0; i < p.splits; i++) {
        const int64_t a = i * p.rows_all + at;
        const float f = __builtin_amdgcn_exp2f(p.part_ml[2 * a] - top);
        sum = __builtin_fmaf(f, p.part_ml[2 * a + 1], sum);
#pragma unroll
        for (int d = 0; d < E; d++)
            acc[d] = __builtin_fmaf(f, p.part_o[a * D + lane * E + d], acc[d]);
    }
    const float f = sum == 0.0f ? 0.0f : p.v_mul / sum;
    const int64_t row = at / p.heads, hd = at - row * p.heads;
    uint16_t* dst = p.out + row * p.o_st + hd * p.o_sh + lane * E;
    if constexpr (E == 1) {
        dst[0] = (uint16_t)pack_bf16(acc[0] * f, 0.0f);
    } else {
#pragma unroll
        for (int d = 0; d < E; d += 2)
            *reinterpret_cast<uint32_t*>(dst + d) = pack_bf16(acc[d] * f, acc[d + 1] * f);
    }
}

// ---------------------------------------------------------------------------
// Host side: which kernel, how many splits.
struct Plan {
    int blocks;  // row blocks of 16 per tile
    int row_tiles;
    int splits;
    int64_t ws_o, ws_ml;  // bytes
};

Plan plan_of(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    Plan pl;
    const int64_t group = a.heads / c.kv_heads, rows = a.max_q * group;
    pl.blocks = rows <= 16 || c.head_dim == 256 ? 1 : 2;
    pl.row_tiles = (int)((rows + 16 * pl.blocks - 1) / (16 * pl.blocks));
    // Splits of the keys: enough workgroups to fill 256 CUs a few times over,
    // and at least one unit for each wave of a split.
    int64_t keys = a.max_len;
    if (a.window && a.window + a.sinks + a.max_q < keys) keys = a.window + a.sinks + a.max_q;
    const int64_t base = a.batch * c.kv_heads * pl.row_tiles;
    const int64_t most = (keys + kUnit * kWaves - 1) / (kUnit * kWaves);
    int64_t s = base > 0 ? 1024 / base : 1;
    s = s > most ? most : s;
    pl.splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
    const int64_t rows_all = a.total_q * a.heads;
    pl.ws_o = pl.splits > 1 ? pl.splits * rows_all * c.head_dim * 4 : 0;
    pl.ws_ml = pl.splits > 1 ? pl.splits * rows_all * 8 : 0;
    return pl;
}

template <int D, int kBlocks>
hipError_t few_rows(const Args& p, hipStream_t stream) {
    constexpr int lds = FewRows<D, kBlocks>::kLds;
    const void* f = (const void*)few_rows_kernel<D, kBlocks>;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const int64_t grid = (int64_t)p.batch_heads * p.row_tiles * p.splits;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((few_rows_kernel<D, kBlocks>), dim3((unsigned)grid), dim3(kThreads), lds,
                       stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t joins = (p.rows_all + kWaves - 1) / kWaves;
    if (joins > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((join_kernel<D>), dim3((unsigned)joins), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

template <int D>
hipError_t dispatch(const Args& p, const Plan& pl, hipStream_t stream) {
    if constexpr (D < 256) {
        if (pl.blocks == 2) return few_rows<D, 2>(p, stream);
    }
    return few_rows<D, 1>(p, stream);
}

int clamp_int(int64_t v) { return (int)(v > 0x3FFFFFFF ? 0x3FFFFFFF : v); }

}  // namespace

int64_t kv_attention_workspace(const if4_kv_cache& c, const if4_kv_attention_args& a) {
    const Plan pl = plan_of(c, a);
    return pl.ws_o + pl.ws_ml;
}

hipError_t launch_kv_attention(const if4_kv_cache& c, const if4_kv_attention_args& a,
                               void* workspace, hipStream_t stream) {
    const Plan pl = plan_of(c, a);
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
    p.part_ml = p.part_o + pl.ws_o / 4;
    p.rows_all = a.total_q * a.heads;
    p.total_q = (int)a.total_q;
    p.pages = (int)c.pages;
    p.kv_heads = (int)c.kv_heads;
    p.heads = (int)a.heads;
    p.group = (int)(a.heads / c.kv_heads);
    p.batch_heads = (int)(a.batch * c.kv_heads);
    p.row_tiles = pl.row_tiles;
    p.splits = pl.splits;
    p.causal = a.causal != 0;
    p.window = clamp_int(a.window);
    p.sinks = clamp_int(a.sinks);
    // n / d = n * ceil(2^(31 + s) / d) >> (31 + s) for n < 2^31 and
    // s = ceil(log2 d): the multiplier exceeds 2^(31 + s) / d by less than
    // 1 <= 2^s / d, which adds less than 1 / d to the quotient
    p.page_tiles = (uint32_t)(c.page_size / 16);
    int sh = 0;
    while (((uint64_t)1 << sh) < p.page_tiles) sh++;
    p.page_shift = 31 + sh;
    p.page_magic = (uint32_t)((((uint64_t)1 << p.page_shift) + p.page_tiles - 1) / p.page_tiles);
    p.q_scale = a.scale * 1.44269504f;
    p.k_exp = c.k_exp + 9;
    p.v_mul = pow2f(c.v_exp + 9);
    if (c.head_dim == 64) return dispatch<64>(p, pl, stream);
    if (c.head_dim == 128) return dispatch<128>(p, pl, stream);
    return dispatch<256>(p, pl, stream);
}

}  // namespace if4
